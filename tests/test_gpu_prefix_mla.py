"""Dense MLA behind a shared prefix on the GPU against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import oracle as O
from paged_helpers import Batch, assert_attention_close, i32, to_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_attention_indexer_head_b200 import build
    build.build()
    from sparse_attention_indexer_head_b200 import binding
    binding.dsa_device_status(reset=True)
    return binding


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("tokens", [1, 2, 31, 32, 33, 64, 257])
def test_one_request_no_prefix(lib, tokens, rope, fp8):
    Batch(tokens, [tokens], page=32, rope=rope, fp8=fp8).run_and_check(lib)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16, 24, 32, 48, 64, 128])
def test_pages_that_end_inside_a_tile(lib, page, fp8):
    Batch(page, [150, 1, 63], prefix=97, page=page, hm=32, fp8=fp8).run_and_check(lib)


@pytest.mark.parametrize("hm", [16, 32, 48, 64, 80, 96, 112, 128])
def test_heads(lib, hm):
    for rope in (0, 64):
        Batch(hm + rope, [40, 3, 70, 129, 5], prefix=64, hm=hm, rope=rope).run_and_check(lib)


@pytest.mark.parametrize("prefix", [1, 15, 32, 33, 500])
def test_prefix_lengths_and_several_queries(lib, prefix):
    # per = 3: the earliest query of a one-token request sits inside the prefix
    for hm in (16, 64):
        Batch(prefix, [1, 90, 2], prefix=prefix, page=16, hm=hm, per=3).run_and_check(lib)


def test_queries_that_see_nothing_or_part_of_the_prefix(lib):
    # requests out of range (padding rows of a captured batch), positions before the first
    # token, inside the prefix, at its end and past the sequence
    for hm in (16, 32, 64, 128):
        Batch(hm, [50, 0, 7], prefix=80, page=16, hm=hm, q_req=[0, -1, 1, 2, 3, 0, 2, 1, 0],
              q_pos=[129, 5, 79, 10 ** 6, 4, -1, 3, 2 ** 31 - 1, 60]).run_and_check(lib)


def test_every_query_empty(lib):
    for hm in (16, 64):
        Batch(1, [0, 0], prefix=0, hm=hm, q_pos=[3, 0]).run_and_check(lib)
        Batch(1, [4], hm=hm, q_req=[7, -3], q_pos=[3, 3]).run_and_check(lib)


def test_missing_pages_and_short_tables(lib):
    b = Batch(3, [200, 90, 64], prefix=48, page=16, hm=16, drop=[(0, 4), (1, 3), (2, 5), (0, 12)])
    b.run_and_check(lib)
    # the table's row ends before the sequence does, and a page lies past the cache
    b = Batch(4, [200, 90], prefix=0, page=16, hm=64)
    b.table[1, 2] = b.rows // 16
    b.table = np.ascontiguousarray(b.table[:, :9])
    b.run_and_check(lib)
    # nothing at all has a page
    b = Batch(5, [40, 33], page=16, hm=32, drop=[(0, 0), (0, 1), (0, 2), (1, 0), (1, 1), (1, 2)])
    b.run_and_check(lib)


def test_prefix_length_beyond_its_pages_is_cut(lib):
    b = Batch(6, [20, 30], prefix=64, page=32, hm=16)
    d, o = b.device(), b.buffers(lib)
    d["prefix_len"] = i32([10 ** 9])           # two pages hold 64 tokens
    b.call(lib, d, o)
    torch.cuda.synchronize()
    b.check(lib, o)
    d["prefix_len"] = i32([-5])                # none: tokens below 64 have no page of their own
    b.call(lib, d, o)
    torch.cuda.synchronize()
    b.P = 0
    b.check(lib, o)


def test_nan_in_one_request_stays_there(lib):
    # four requests share a tile of rows; request 1 holds a NaN and request 2 an infinity
    b = Batch(7, [70, 64, 33, 90], prefix=40, page=16, hm=16)
    clean = b.oracle()
    for req, t, bad in [(1, 50, np.nan), (2, 41, np.inf)]:
        b.values[O.paged_row(b.table[req], 16, t, b.rows), 300] = bad
    d, o = b.device(), b.buffers(lib)
    b.call(lib, d, o)
    torch.cuda.synchronize()
    out, lse = o["out"].float().cpu().numpy(), o["lse"].cpu().numpy()
    keep = [0, 3]
    assert_attention_close(out[keep], lse[keep], [x[keep] for x in clean], b.width)
    assert np.isnan(out[1]).any() and not np.isfinite(out[2]).all()


def test_large_and_negative_logits(lib):
    # scaled so that logits reach a few hundred: the running maximum moves and rows rescale
    b = Batch(8, [400, 300], prefix=333, page=16, hm=64, spread=20.0)
    b.run_and_check(lib)
    b = Batch(9, [100, 40], prefix=64, page=32, hm=32)
    b.sm_scale = -b.sm_scale
    b.run_and_check(lib)
    b.sm_scale = 0.0
    b.run_and_check(lib)


@pytest.mark.parametrize("own", [40, 5000])              # one part, and parts that are merged
def test_infinite_logits(lib, own):
    # channel 9 of every row is 1: head 1's logits are all -infinity, head 2's all +infinity
    b = Batch(26, [own], page=32, hm=16, rope=0)
    b.values[:, 9] = 1.0
    clean = b.oracle()
    b.q[0, 1, 9], b.q[0, 2, 9] = -np.inf, np.inf
    d, o = b.device(), b.buffers(lib)
    b.call(lib, d, o)
    torch.cuda.synchronize()
    out, lse = o["out"].float().cpu().numpy(), o["lse"].cpu().numpy()
    rest = [h for h in range(16) if h not in (1, 2)]
    assert_attention_close(out[:, rest], lse[:, rest], [x if i == 4 else x[:, rest] for i, x in enumerate(clean)], b.width)
    assert (out[0, 1] == 0).all() and np.isneginf(lse[0, 1])
    assert np.isnan(out[0, 2]).all() and np.isnan(lse[0, 2])


def test_rows_that_grow_along_the_sequence(lib):
    # every later token has a larger logit: each tile raises the maximum of every row
    b = Batch(10, [700], prefix=0, page=64, hm=64, rope=0)
    b.q[:] = np.abs(b.q)
    for t in range(700):
        b.values[O.paged_row(b.table[0], 64, t, b.rows)] = np.float32(t // 4) / 16
    b.run_and_check(lib)


def test_long_sequence_in_parts(lib):
    for hm, rope, fp8 in [(16, 0, False), (128, 64, False), (32, 64, True)]:
        Batch(hm, [9001], prefix=1003, page=64, hm=hm, rope=rope, fp8=fp8).run_and_check(lib)


def test_many_ragged_requests(lib):
    rng = np.random.default_rng(5)
    own = [int(x) for x in rng.integers(0, 300, 150)]
    Batch(11, own, prefix=129, page=32, hm=16).run_and_check(lib)
    Batch(12, own[:60], prefix=0, page=16, hm=64, rope=0).run_and_check(lib)
    Batch(13, own[:40], prefix=70, page=24, hm=128, fp8=True).run_and_check(lib)


def test_rows_past_two_to_the_32_bytes(lib):
    # a cache of 4.4 GB whose used pages lie at its end
    rows, page = 4_300_800, 64
    b = Batch(14, [100, 65], prefix=64, page=page, hm=16, rope=0)
    big = torch.empty(rows, 512, dtype=torch.bfloat16, device="cuda")
    d, o = b.device(), b.buffers(lib)
    shift = rows // page - b.rows // page
    big[shift * page:] = d["cache"]
    d["cache"] = big
    for k in ("table", "prefix_table"):
        d[k] = torch.where(d[k] >= 0, d[k] + shift, d[k])
    small, b.rows = b.rows, rows
    b.call(lib, d, o)
    torch.cuda.synchronize()
    b.rows = small
    b.check(lib, o)


def test_results_are_the_same_bits_every_time(lib):
    b = Batch(15, [2000, 31, 700, 1], prefix=515, page=32, hm=32)
    d, o = b.device(), b.buffers(lib)
    b.call(lib, d, o)
    p = b.buffers(lib)
    p["ws"].zero_()
    b.call(lib, d, p)
    torch.cuda.synchronize()
    assert torch.equal(o["out"], p["out"]) and torch.equal(o["lse"], p["lse"])
    b.check(lib, o)


def test_no_lse_and_nothing_written_past_the_outputs(lib):
    b = Batch(16, [60, 90, 4], prefix=32, hm=48)
    d, o = b.device(), b.buffers(lib)
    room = torch.full((b.Q + 2, b.hm, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    need = lib.dsa_prefix_mla_workspace_size(b.Q, b.hm)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    want = b.buffers(lib)
    b.call(lib, d, want)
    o["out"], o["lse"], o["ws"] = room[1:-1], None, ws[:need]
    b.call(lib, d, o)
    torch.cuda.synchronize()
    assert torch.equal(room[1:-1], want["out"])
    assert (room[0] == 7).all() and (room[-1] == 7).all() and (ws[need:] == 0x5A).all()


def test_captured_call_replays_over_other_lengths(lib):
    # unowned rows are 0 here: with 187 shared tokens the requests' own pages hold rows 192 .. 199
    b = Batch(17, [300, 129, 64, 17], prefix=200, page=16, hm=16, fill=0.0)
    d, o = b.device(), b.buffers(lib)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        b.call(lib, d, o, s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        b.call(lib, d, o, s)
    for own, P in [([300, 129, 64, 17], 200), ([1, 128, 3, 0], 200), ([250, 60, 0, 9], 187)]:
        # 187: the last tokens of the prefix's pages become each request's own, in no page of
        # its own where the table has none
        b.seq_len = np.asarray([200 + n for n in own], np.int32)
        b.q_pos, b.P = b.seq_len - 1, P
        d["seq_len"].copy_(i32(b.seq_len))
        d["q_pos"].copy_(i32(b.q_pos))
        d["prefix_len"].fill_(P)
        o["out"].fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        b.check(lib, o)


def test_two_streams_with_a_workspace_each(lib):
    a, b = Batch(18, [900, 30], prefix=64, hm=64), Batch(19, [500, 700, 9], prefix=31, hm=16)
    da, oa, db, ob = a.device(), a.buffers(lib), b.device(), b.buffers(lib)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        a.call(lib, da, oa, s)
        b.call(lib, db, ob, t)
    torch.cuda.synchronize()
    a.check(lib, oa)
    b.check(lib, ob)


def test_back_to_back_calls_on_one_stream_share_a_workspace(lib):
    # the second call's partial results must not overtake the first call's merge
    a, b = Batch(20, [4000], hm=64), Batch(21, [3500], hm=64)
    da, oa, db, ob = a.device(), a.buffers(lib), b.device(), b.buffers(lib)
    ob["ws"] = oa["ws"]
    for _ in range(10):
        a.call(lib, da, oa)
        b.call(lib, db, ob)
    torch.cuda.synchronize()
    a.check(lib, oa)
    b.check(lib, ob)


def test_equals_the_sparse_call_on_every_token(lib):
    # NoPE: the sparse paged MLA over all ids is the dense call; both within their tolerance
    b = Batch(22, [200, 64], prefix=0, page=16, hm=64, rope=0)
    d, o = b.device(), b.buffers(lib)
    b.call(lib, d, o)
    ids = i32(np.where(np.arange(256) < b.seq_len[:, None], np.arange(256), -1))
    ws = torch.empty(max(16, lib.dsa_sparse_mla_workspace_size(b.Q, 64, 256)), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(o["out"]), torch.empty_like(o["lse"])
    lib.dsa_sparse_mla_decode_paged(d["q"], d["cache"], b.rows, d["table"], b.table.shape[1], 16, d["seq_len"],
                                    d["q_req"], ids, b.Q, b.B, 64, 256, 512, 0, b.sm_scale, out, lse, ws, ws.numel())
    torch.cuda.synchronize()
    b.check(lib, o)
    ref, rlse, mag, _, _ = b.oracle()
    # the sparse call's weights and its parts are bf16: one rounding of each more
    tol = 2.0 ** -8 * np.abs(ref) + (2 * 2.0 ** -8 + 2.0 ** -12) * mag
    assert (np.abs(out.float().cpu().numpy() - ref) <= tol).all()
    assert np.abs(lse.cpu().numpy() - o["lse"].cpu().numpy()).max() < 1e-4


def test_every_fp8_code(lib):
    # rows of all 256 codes, NaN codes among them: values are exact, and a NaN shows where it lies
    for rope in (0, 64):
        b = Batch(23, [40, 64], prefix=0, page=32, hm=16, rope=rope, fp8=True, fill=0.0, scale=0.5)
        rng = np.random.default_rng(1)
        b.codes[:] = rng.integers(0, 256, b.codes.shape)
        b.codes[(b.codes & 0x7F) == 0x7F] = 0x80
        b.values = O.e4m3_to_f64(b.codes) * 0.5
        b.q *= np.float32(2.0 ** -6)                  # codes reach 448
        d, o = b.run_and_check(lib)
        row = O.paged_row(b.table[0], 32, 5, b.rows)
        d["cache"][row, 77], d["cache"][row, 300] = 0x7F, 0xFF
        b.call(lib, d, o)
        torch.cuda.synchronize()
        out = o["out"].float()
        assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("hm", [16, 32])
@pytest.mark.parametrize("prefix", [0, 45])
def test_several_queries_of_one_request_share_a_walk(lib, hm, prefix):
    # runs of two to four queries, runs broken by a padding row or an empty query, equal
    # positions, positions far apart, and a run that ends at a unit's border
    q_req = [0, 0, 0, 1, 2, 2, -1, 2, 0, 1, 1, 1, 1, 3, 3, 2, 2, 2, 2, 2]
    own = [300, 100, 64, 33]
    pos = [299, 10, 150, 99, 63, 63, 5, 31, 32, 96, 97, 98, 99, -50, 20, 63, 62, 32, 31, 0]
    b = Batch(hm, own, prefix=prefix, page=16, hm=hm, q_req=q_req, q_pos=[p + prefix for p in pos])
    b.run_and_check(lib)


def test_a_later_draft_tokens_nan_stays_with_it(lib):
    # token 70 is seen by the second query alone
    b = Batch(24, [71], page=16, hm=16, per=2)
    clean = b.oracle()
    b.values[O.paged_row(b.table[0], 16, 70, b.rows), 5] = np.nan
    d, o = b.device(), b.buffers(lib)
    b.call(lib, d, o)
    torch.cuda.synchronize()
    out, lse = o["out"].float().cpu().numpy(), o["lse"].cpu().numpy()
    assert_attention_close(out[:1], lse[:1], [x[:1] for x in clean], b.width)
    assert np.isnan(out[1]).all()


@pytest.mark.parametrize("requests,hm,lo,hi", [
    (40, 64, 1100, 1900),      # fewer row tiles than CTAs, ranges that cross tiles
    (7, 64, 1, 4000),          # whole CTAs for ragged tiles, some tiles of one unit
    (148, 64, 30, 70),         # a CTA for every tile
    (149, 64, 60, 130),        # one tile more than CTAs: ranges that cross tiles, entries by CTA
    (230, 128, 1, 60),         # two tiles a query, more tiles than a block has threads
    (1000, 16, 0, 3),          # tiles of four queries, many of them empty
])
def test_plans(lib, requests, hm, lo, hi):
    rng = np.random.default_rng(requests)
    own = [int(x) for x in rng.integers(lo, hi + 1, requests)]
    own[-1] = hi
    Batch(requests, own, prefix=0, page=32, hm=hm, rope=0).run_and_check(lib)


def test_a_long_request_among_short_ones(lib):
    for hm in (16, 64):
        Batch(25, [3, 9000, 1, 40] + [5] * 200, prefix=0, page=64, hm=hm, rope=0).run_and_check(lib)


@pytest.mark.parametrize("rope", [0, 64])
@pytest.mark.parametrize("page", [24, 64])
def test_fp8_ring_over_many_row_tiles(lib, page, rope):
    # more row tiles than CTAs: a CTA's stages and slots turn over across parts of many lengths,
    # among them requests without a token of their own
    rng = np.random.default_rng(rope + page)
    own = [int(x) for x in rng.integers(0, 700, 90)]
    Batch(27, own, prefix=100, page=page, hm=128, rope=rope, fp8=True).run_and_check(lib)


def block_threads(fp8):
    """Threads of the attention's block, by the source: the plan takes a row tile a thread."""
    import re
    from sparse_attention_indexer_head_b200 import build
    with open(f"{build.CSRC}/prefix_mla.cuh") as f:
        return int(re.search(r"pm_threads\(bool fp8\) \{ return fp8 \? (\d+) : (\d+);", f.read())[1 if fp8 else 2])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hm,lo,hi", [(128, 0, 60), (64, 1, 40), (16, 0, 9)])
def test_plans_of_more_row_tiles_than_threads(lib, hm, lo, hi, fp8):
    tiles = block_threads(fp8) + 70
    requests = tiles // 2 if hm == 128 else tiles if hm == 64 else 4 * tiles
    rng = np.random.default_rng(hm + fp8)
    own = [int(x) for x in rng.integers(lo, hi + 1, requests)]
    own[3], own[requests // 2] = 1500, 700                  # ranges that end inside a long tile
    Batch(requests, own, page=32, hm=hm, rope=0, fp8=fp8).run_and_check(lib)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hm,n", [(128, 300), (64, 190), (32, 130), (16, 263)])
def test_a_prompt_chunk(lib, hm, n, fp8):
    """Consecutive queries of one request behind a prefix, each seeing one token more than the one
    before, and padding rows behind the last: up to 600 row tiles, or runs of queries that walk
    together."""
    own, P, pad = 20 + n, 75, 5
    q_req = np.r_[np.zeros(n, int), np.full(pad, -1)]
    q_pos = np.r_[P + own - n + np.arange(n), np.zeros(pad, int)]
    Batch(n + hm, [own], prefix=P, page=16, hm=hm, fp8=fp8, q_req=q_req, q_pos=q_pos).run_and_check(lib)


@pytest.mark.parametrize("fp8", [False, True])
def test_the_largest_batch(lib, fp8):
    """65535 queries of 128 heads, each a request of up to three tokens: outputs of 8 GB. Against
    the formula in 64 bits on the device, with assert_attention_close's tolerances."""
    Q, hm, rows, most, scale = 65535, 128, 4096, 3, 0.25
    gen = torch.Generator(device="cuda").manual_seed(5)
    sm = float(np.float32(512 ** -0.5))
    values = torch.randn(rows, 512, generator=gen, device="cuda")
    cache = values.to(torch.float8_e4m3fn) if fp8 else values.to(torch.bfloat16)
    values = cache.double() * (scale if fp8 else 1.0)
    table = torch.randint(0, rows, (Q, most), generator=gen, device="cuda", dtype=torch.int32)
    seq = torch.randint(0, most + 1, (Q,), generator=gen, device="cuda", dtype=torch.int32)
    q = torch.empty(Q, hm, 512, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    out = torch.full((Q, hm, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((Q, hm), float("nan"), device="cuda")
    ws = torch.empty(lib.dsa_prefix_mla_workspace_size(Q, hm), dtype=torch.uint8, device="cuda")
    where = (None, 0, None, table, most, 1, seq, torch.arange(Q, dtype=torch.int32, device="cuda"), seq - 1, Q, Q, hm, 512, 0,
             sm, out, lse, ws, ws.numel())
    if fp8:
        lib.dsa_prefix_mla_decode_paged_fp8(q, cache.view(torch.uint8), scale, rows, *where)
    else:
        lib.dsa_prefix_mla_decode_paged(q, cache, rows, *where)
    torch.cuda.synchronize()
    assert lib.dsa_device_status(reset=True) == 0
    token = torch.arange(most, device="cuda")
    for i in range(0, Q, 2048):
        k, x, n = values[table[i:i + 2048].long()], q[i:i + 2048].double(), seq[i:i + 2048]
        seen = (token < n[:, None])[:, None]
        z = (x @ k.transpose(1, 2) * sm).masked_fill(~seen, -np.inf)
        terms = (x.abs() @ k.abs().transpose(1, 2) * sm).masked_fill(~seen, 0).amax(2)
        p = torch.where(n[:, None, None] > 0, torch.softmax(z, 2), 0.0)
        ref, rlse, mag = p @ k, torch.logsumexp(z, 2), p @ k.abs()
        dz = (512 + 12) * 2.0 ** -23 * terms + 2.0 ** -21
        sums = (n[:, None] + 8) * 2.0 ** -23
        tol = (2.0 ** -8 * ref.abs() + mag * (2.0 ** -8 + 2 * dz + 2 * sums)[..., None]) * (1 + 2.0 ** -6)
        assert ((out[i:i + 2048].double() - ref).abs() <= tol).all()
        got, none = lse[i:i + 2048].double(), (n == 0)[:, None].expand(-1, hm)
        assert (torch.isneginf(got) == none).all()
        assert ((got - rlse).abs() <= dz + sums + 2.0 ** -22 * rlse.abs())[~none].all()

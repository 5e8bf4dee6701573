"""The paged latent append on the GPU against the oracle in 64 bits, and the step it belongs to:
append, then the MLA that reads the pages."""
import numpy as np
import pytest
import torch

import oracle as O
from paged_helpers import (Batch, HALF_BF16, HALF_E4M3, SUB_E4M3, assert_attention_close, bf16_round,
                           cos_sin_table, i32, scatter_pages, to_bf16)

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


class Append:
    """New tokens of several requests: request b's tokens first[b] .. first[b] + counts[b] - 1."""

    def __init__(self, seed, counts, first, page=16, rope=64, hm=16, interleaved=True, fp8=False, norm=True,
                 scale=0.125, pad=24, big=1.0):
        rng = np.random.default_rng(seed)
        self.page, self.rope, self.hm, self.interleaved, self.fp8 = page, rope, hm, interleaved, fp8
        self.scale, self.width, self.B, self.pad = scale, 512 + rope, len(counts), pad
        self.table, pages = scatter_pages([f + c for f, c in zip(first, counts)], page, rng)
        self.rows = pages * page
        self.req = np.concatenate([np.full(c, b) for b, c in enumerate(counts)]).astype(np.int32)
        self.pos = np.concatenate([f + np.arange(c) for f, c in zip(first, counts)]).astype(np.int32)
        self.n = len(self.req)
        self.joint = bf16_round(rng.standard_normal((self.n, pad + self.width)) * big)
        self.norm = bf16_round(1 + 0.1 * rng.standard_normal(512)) if norm else None
        self.cos_sin = cos_sin_table(max(1, int(self.pos.max(initial=0)) + 1)) if rope else None
        self.q_wide = bf16_round(rng.standard_normal((self.n, hm, 128 + rope)))

    def device(self):
        old = torch.randn(self.rows, self.width, device="cuda").to(torch.bfloat16)
        cache = torch.randint(0, 120, old.shape, dtype=torch.uint8, device="cuda") if self.fp8 else old
        return dict(joint=to_bf16(self.joint), norm=None if self.norm is None else to_bf16(self.norm),
                    cos_sin=None if self.cos_sin is None else torch.from_numpy(self.cos_sin).cuda(),
                    req=i32(self.req), pos=i32(self.pos), table=i32(self.table), cache=cache,
                    q_wide=to_bf16(self.q_wide),
                    q=torch.randn(self.n, self.hm, self.width, device="cuda").to(torch.bfloat16))

    def call(self, lib, d, heads=True, stream=None):
        heads = heads and self.rope > 0
        shape = (d["joint"].stride(0), d["norm"], 1e-5, d["cos_sin"], 0 if self.cos_sin is None else len(self.cos_sin),
                 int(self.interleaved), d["req"], d["pos"], self.n, 512, self.rope, d["table"], self.B,
                 self.table.shape[1], self.page)
        queries = (d["q_wide"][..., 128:], d["q_wide"].stride(0), d["q_wide"].stride(1), self.hm, d["q"]) if heads else ()
        if self.fp8:
            lib.dsa_latent_append_paged_fp8(d["joint"][:, self.pad:], *shape, d["cache"], self.scale, self.rows,
                                            *queries, stream=stream)
        else:
            lib.dsa_latent_append_paged(d["joint"][:, self.pad:], *shape, d["cache"], self.rows, *queries, stream=stream)

    def oracle(self):
        return O.latent_append(self.joint[:, self.pad:], self.norm, 1e-5, self.cos_sin, self.interleaved, self.req,
                               self.pos, self.table, self.page, self.rows, self.q_wide[..., 128:] if self.rope else None)

    def run_and_check(self, lib, heads=True):
        d = self.device()
        before, q_before = d["cache"].clone(), d["q"].clone()
        self.call(lib, d, heads)
        torch.cuda.synchronize()
        self.check(d, before, q_before, heads)
        return d

    def check(self, d, before, q_before, heads=True):
        rows, turned = self.oracle()
        at = sorted(rows)
        new = d["cache"][at]
        if at:
            assert_rows_close(new, np.stack([rows[r] for r in at]), self)
        keep = torch.ones(self.rows, dtype=torch.bool)
        keep[at] = False
        assert torch.equal(d["cache"][keep.cuda()].view(torch.uint8), before[keep.cuda()].view(torch.uint8))
        assert torch.equal(d["q"][..., :512], q_before[..., :512])
        got = d["q"][..., 512:].float().cpu().numpy()
        for i in range(self.n if self.rope else 0):
            if heads and i in turned:
                x = np.abs(self.q_wide[i, :, 128:]).astype(np.float64)
                # a pair's result: two products and one addition in fp32, then bf16
                size = x + (np.roll(x, 32, -1) if not self.interleaved else x.reshape(-1, 32, 2)[..., ::-1].reshape(x.shape))
                assert (np.abs(got[i] - turned[i]) <= HALF_BF16 * np.abs(turned[i]) + 2.0 ** -21 * size).all()
            else:
                assert torch.equal(d["q"][i], q_before[i])


def assert_rows_close(new, want, a):
    """A stored value is off by half a step of its type, after fp32 arithmetic: the mean of 512
    squares (22 additions deep: 2^-20 relative), its reciprocal root and two or three products
    (2^-21 together), or a pair's two products and their sum (2^-22 of the terms, which are at
    most the pair's length: 8 standard deviations here)."""
    soft = 2.0 ** -19
    if a.fp8:
        got = O.e4m3_to_f64(new.cpu().numpy())
        want = np.clip(want / a.scale, -448, 448)
        size = 8 * 2.0 ** -21 / a.scale
        tol = np.maximum(HALF_E4M3 * np.abs(want), SUB_E4M3) * (1 + soft) + soft * np.abs(want) + size
    else:
        got = new.float().cpu().numpy()
        tol = HALF_BF16 * np.abs(want) * (1 + soft) + soft * np.abs(want) + 8 * 2.0 ** -21 * max(1.0, np.abs(want).max() / 8)
    err = np.abs(got - want)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} values outside, worst {np.nanmax(err - tol):.3g} over"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("hm", [1, 16, 40, 128])
def test_rotated(lib, hm, interleaved, fp8):
    Append(hm, [1, 5, 33], [0, 100, 7], hm=hm, interleaved=interleaved, fp8=fp8).run_and_check(lib)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
def test_nope_and_pages(lib, page, fp8):
    Append(page, [1, 40, 3], [2, 0, 130], page=page, rope=0, fp8=fp8).run_and_check(lib)
    Append(page, [3, 1], [2, 64], page=page, fp8=fp8, norm=False).run_and_check(lib, heads=False)


def test_many_tokens(lib):
    Append(1, [700, 1, 333], [0, 5000, 90], hm=32).run_and_check(lib)


def test_saturation_and_zero_rows(lib):
    a = Append(2, [6], [3], fp8=True, norm=False, scale=0.01, big=3.0)
    a.joint[2] = 0
    a.run_and_check(lib)
    b = Append(2, [6], [3])
    b.joint[2] = 0                                 # mean square 0: eps carries the root
    b.run_and_check(lib)


def test_nan_and_infinity_stay_in_their_row(lib):
    for fp8 in (False, True):
        a = Append(4, [5], [0], fp8=fp8, norm=False)
        d = a.device()
        want = a.device()
        for k in ("cache", "q"):
            want[k].copy_(d[k])
        a.call(lib, want)
        d["joint"][2, a.pad + 9] = float("nan")
        d["joint"][3, a.pad + 8] = float("-inf")
        a.call(lib, d)
        torch.cuda.synchronize()
        at = [O.paged_row(a.table[0], a.page, t, a.rows) for t in range(5)]
        c = d["cache"].view(torch.float8_e4m3fn).float() if fp8 else d["cache"].float()
        assert torch.isnan(c[at[2], 9]) and c[at[3], 8] == (-448.0 if fp8 else -float("inf"))
        same = (d["cache"] == want["cache"]).cpu()
        same[at[2], 9] = same[at[3], 8] = True
        assert same.all()


def test_tokens_that_are_skipped(lib):
    a = Append(5, [4, 4, 4], [0, 16, 40])
    a.req[1], a.req[5] = -1, 3                     # requests outside the batch
    a.pos[2], a.pos[6] = -1, 10 ** 6               # before the first token, past the table of positions
    a.table[2, 2] = -1                             # a missing page: heads alone
    a.run_and_check(lib)
    b = Append(6, [20, 20], [0, 0], rope=0)
    b.table = np.ascontiguousarray(b.table[:, :1])  # tokens past the table's row
    b.table[1, 0] = b.rows // b.page               # a page past the cache
    b.run_and_check(lib)


def test_rotation_in_place(lib):
    a = Append(7, [9, 2], [0, 30], interleaved=False)
    d = a.device()
    ref = a.device()
    a.call(lib, ref)
    d["q"][..., 512:] = d["q_wide"][..., 128:]
    head = d["q"][..., :512].clone()
    lib.dsa_latent_append_paged(d["joint"][:, a.pad:], d["joint"].stride(0), d["norm"], 1e-5, d["cos_sin"], len(a.cos_sin),
                                0, d["req"], d["pos"], a.n, 512, 64, d["table"], a.B, a.table.shape[1], a.page, d["cache"],
                                a.rows, d["q"][..., 512:], d["q"].stride(0), d["q"].stride(1), a.hm, d["q"])
    torch.cuda.synchronize()
    assert torch.equal(d["q"][..., 512:], ref["q"][..., 512:]) and torch.equal(d["q"][..., :512], head)


def test_far_positions(lib):
    # angles at positions near 2^20: the table's, not a product in 32 bits
    a = Append(8, [3], [(1 << 20) - 3], page=64, hm=16)
    a.run_and_check(lib)


def test_rows_past_two_to_the_32_bytes(lib):
    a = Append(9, [3, 2], [0, 70], page=64, rope=0)
    d = a.device()
    big = torch.zeros(4_300_800, 512, dtype=torch.bfloat16, device="cuda")
    shift = 4_300_800 // 64 - a.rows // 64
    big[shift * 64:] = d["cache"]
    before = d["cache"].clone()
    d["cache"], small = big, a.rows
    d["table"] = torch.where(d["table"] >= 0, d["table"] + shift, d["table"])
    a.rows = big.shape[0]
    a.call(lib, d)
    torch.cuda.synchronize()
    a.rows, d["cache"] = small, big[shift * 64:]
    a.check(d, before, d["q"].clone())
    assert not big[:shift * 64].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_steps_behind_a_prefix(lib, fp8):
    """Append, then the MLA over what was appended, captured once and replayed for three steps;
    the batch is padded with rows whose request is -1."""
    rng = np.random.default_rng(1)
    page, hm, P, B, pad, scale = 16, 16, 53, 5, 2, 0.0625
    n, width, most = B + pad, 576, 40
    whole = P // page
    both, pages = scatter_pages([P] + [P - whole * page + most] * B, page, rng)
    table = np.concatenate([np.full((B, whole), -1), both[1:]], 1).astype(np.int32)
    rows = pages * page
    own = np.array([0, 1, 11, 12, 37])
    values = bf16_round(rng.standard_normal((rows, width)))
    if fp8:
        codes = rng.integers(0, 0x58, values.shape).astype(np.uint8)
        values = O.e4m3_to_f64(codes) * scale
    cache = torch.from_numpy(codes).cuda() if fp8 else to_bf16(values)
    cs = cos_sin_table(P + most)
    w = bf16_round(1 + 0.1 * rng.standard_normal(512))
    dev = dict(w=to_bf16(w), cs=torch.from_numpy(cs).cuda(), table=i32(table), prefix=i32(both[0]), plen=i32([P]),
               req=i32(np.r_[np.arange(B), [-1] * pad]), pos=i32(np.zeros(n)), seq=i32(np.zeros(B)))
    new = torch.zeros(n, width, dtype=torch.bfloat16, device="cuda")
    q_rot = torch.zeros(n, hm, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(n, hm, width, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(n, hm, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, hm, device="cuda")
    ws = torch.empty(lib.dsa_prefix_mla_workspace_size(n, hm), dtype=torch.uint8, device="cuda")
    sm = float(np.float32(width ** -0.5))

    def step(stream):
        a = (dev["w"], 1e-6, dev["cs"], len(cs), 1, dev["req"], dev["pos"], n, 512, 64, dev["table"], B, table.shape[1], page)
        h = (q_rot, hm * 64, 64, hm, q)
        m = (dev["prefix"], len(both[0]), dev["plen"], dev["table"], table.shape[1], page, dev["seq"], dev["req"], dev["pos"],
             n, B, hm, 512, 64, sm, out, lse, ws, ws.numel(), stream)
        if fp8:
            lib.dsa_latent_append_paged_fp8(new, width, *a, cache, scale, rows, *h, stream=stream)
            lib.dsa_prefix_mla_decode_paged_fp8(q, cache, scale, rows, *m)
        else:
            lib.dsa_latent_append_paged(new, width, *a, cache, rows, *h, stream=stream)
            lib.dsa_prefix_mla_decode_paged(q, cache, rows, *m)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(s)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        step(s)
    for _ in range(3):
        x = bf16_round(rng.standard_normal((n, width)) * 2)
        heads = bf16_round(rng.standard_normal((n, hm, 64)))
        lat = bf16_round(rng.standard_normal((n, hm, 512)))
        pos = np.r_[P + own, [0] * pad]
        new.copy_(to_bf16(x))
        q_rot.copy_(to_bf16(heads))
        q[..., :512] = to_bf16(lat)
        dev["pos"].copy_(i32(pos))
        dev["seq"].copy_(i32(P + own + 1))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert lib.dsa_device_status(reset=True) == 0
        # each stage against the oracle on the stage's own inputs
        added, turned = O.latent_append(x, w, 1e-6, cs, True, np.r_[np.arange(B), [-1] * pad], pos, table, page, rows, heads)
        assert len(added) == B and sorted(turned) == list(range(B))
        stored = O.e4m3_to_f64(cache.cpu().numpy()) * scale if fp8 else cache.float().cpu().numpy().astype(np.float64)
        for r, y in added.items():
            step_size = np.maximum(HALF_E4M3 * np.abs(y), SUB_E4M3 * scale) if fp8 else HALF_BF16 * np.abs(y)
            # half a step, and fp32 arithmetic: 2^-22 of a pair's two terms, each below 10
            assert (np.abs(stored[r] - y) <= step_size * (1 + 2.0 ** -18) + 2.0 ** -17).all()
            values[r] = stored[r]
        np.testing.assert_array_equal(stored, values)          # and no other row moved
        want = O.prefix_mla(q.float().cpu().numpy(), values, both[0], P, table, page, P + own + 1,
                            np.r_[np.arange(B), [-1] * pad], pos, sm)
        assert_attention_close(out.float().cpu().numpy(), lse.cpu().numpy(), want, width)
        own = own + 1


@pytest.mark.parametrize("fp8", [False, True])
def test_append_then_sparse_mla(lib, fp8):
    """NoPE rows appended to pages are what the sparse paged MLA reads."""
    a = Append(10, [70, 33], [0, 0], rope=0, page=16, fp8=fp8)
    d = a.device()
    a.call(lib, d)
    q = bf16_round(np.random.default_rng(2).standard_normal((2, 16, 512)))
    dq, seq, W_ = to_bf16(q), i32([70, 33]), 64
    ids = np.stack([np.random.default_rng(3).permutation(70)[:W_], np.r_[np.arange(33), [-1] * 31]]).astype(np.int32)
    out = torch.empty(2, 16, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 16, device="cuda")
    ws = torch.empty(max(16, lib.dsa_sparse_mla_workspace_size(2, 16, W_)), dtype=torch.uint8, device="cuda")
    tail = (a.rows, d["table"], a.table.shape[1], 16, seq, i32([0, 1]), i32(ids), 2, 2, 16, W_, 512, 0, 512 ** -0.5, out, lse,
            ws, ws.numel())
    if fp8:
        lib.dsa_sparse_mla_decode_paged_fp8(dq, d["cache"], a.scale, *tail)
    else:
        lib.dsa_sparse_mla_decode_paged(dq, d["cache"], *tail)
    torch.cuda.synchronize()
    stored = O.e4m3_to_f64(d["cache"].cpu().numpy()) * a.scale if fp8 else d["cache"].float().cpu().numpy()
    for i, T in enumerate([70, 33]):
        rows = [O.paged_row(a.table[i], 16, int(t), a.rows) for t in ids[i] if 0 <= t < T]
        k = stored[rows].astype(np.float64)
        z = q[i] @ k.T * 512 ** -0.5
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        tol = 2.0 ** -8 * np.abs(p @ k) + (2 * 2.0 ** -8 + 2.0 ** -12) * (p @ np.abs(k))
        assert (np.abs(out[i].float().cpu().numpy() - p @ k) <= tol).all()


@pytest.mark.parametrize("fp8,rope,graph", [(False, 64, True), (True, 64, False), (False, 0, False), (True, 0, True)])
def test_pipeline_prefix_decode(lib, fp8, rope, graph):
    """pipeline.PrefixDecode: the prefix filled once, then steps, against the oracle end to end:
    each step's output for the rows that the cache holds."""
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    rng = np.random.default_rng(rope + fp8)
    R, hm, P, page, scale, width = 3, 32, 37, 16, 0.0625, 512 + rope
    w = bf16_round(1 + 0.1 * rng.standard_normal(512))
    cs = cos_sin_table(64, rope) if rope else None
    dec = PrefixDecode(R, hm, 20, P, norm_w=torch.from_numpy(w), cos_sin=None if cs is None else torch.from_numpy(cs),
                       page=page, fp8=fp8, kv_scale=scale if fp8 else 1.0, graph=graph, sm_scale=width ** -0.5)
    x = bf16_round(rng.standard_normal((P, width)))
    dec.fill_prefix(to_bf16(x))
    prefix, table = dec.prefix_table.cpu().numpy(), dec.block_table.cpu().numpy()
    rows, _ = O.latent_append(x, w, 1e-6, cs, True, np.zeros(P, int), np.arange(P), prefix[None], page, dec.kv_rows)

    def stored():
        c = dec.cache.cpu()
        return O.e4m3_to_f64(c.numpy()) * scale if fp8 else c.float().numpy().astype(np.float64)

    def check(rows):
        kv = stored()
        for r, y in rows.items():
            half = np.maximum(HALF_E4M3 * np.abs(y), SUB_E4M3 * scale) if fp8 else HALF_BF16 * np.abs(y)
            assert (np.abs(kv[r] - y) <= half * (1 + 2.0 ** -18) + 2.0 ** -17).all()
        return kv

    check(rows)
    for t in range(3):
        x = bf16_round(rng.standard_normal((R, width)))
        q = bf16_round(rng.standard_normal((R, hm, width)))
        out = dec.step(to_bf16(x), to_bf16(q)).float().cpu().numpy()
        assert lib.dsa_device_status(reset=True) == 0
        pos = np.full(R, P + t)
        rows, heads = O.latent_append(x, w, 1e-6, cs, True, np.arange(R), pos, table, page, dec.kv_rows,
                                      q[..., 512:] if rope else None)
        assert len(rows) == R
        kv = check(rows)
        turned = dec.q.float().cpu().numpy()
        np.testing.assert_array_equal(turned[..., :512], q[..., :512])
        for i, y in heads.items():
            # half a step, and 2^-22 of a pair's two terms, each below 10
            assert (np.abs(turned[i, :, 512:] - y) <= HALF_BF16 * np.abs(y) * (1 + 2.0 ** -18) + 2.0 ** -17).all()
        want = O.prefix_mla(turned, kv, prefix, P, table, page, pos + 1, np.arange(R), pos, width ** -0.5)
        assert_attention_close(out, dec.lse.cpu().numpy(), want, width)


def test_pipeline_prefix_decode_refuses(lib):
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    with pytest.raises(ValueError):
        PrefixDecode(1, 16, 8, 60, norm_w=None, cos_sin=torch.zeros(64, 64))        # 68 positions
    dec = PrefixDecode(1, 16, 1, 4, norm_w=None)
    with pytest.raises(ValueError):
        dec.fill_prefix(torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda"))
    dec.fill_prefix(torch.zeros(4, 512, dtype=torch.bfloat16, device="cuda"))
    row = torch.zeros(1, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 16, 512, dtype=torch.bfloat16, device="cuda")
    dec.step(*row)
    with pytest.raises(ValueError):
        dec.step(*row)


def test_pipeline_prefix_decode_refuses_other_shapes(lib):
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    dec = PrefixDecode(2, 16, 4, 4, norm_w=None)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):                     # the channels of a row apart
        dec.fill_prefix(torch.zeros(512, 4, **bf).t())
    with pytest.raises(ValueError):
        dec.fill_prefix(torch.zeros(4, 512, device="cuda"))
    with pytest.raises(ValueError):
        dec.fill_prefix(torch.zeros(4, 512, dtype=torch.bfloat16))
    kv_new, q = torch.zeros(2, 512, **bf), torch.zeros(2, 16, 512, **bf)
    for bad in [(kv_new[:1], q), (kv_new, q[:, :1]), (kv_new, q[0]), (kv_new.float(), q), (kv_new, q.half())]:
        with pytest.raises(ValueError):
            dec.step(*bad)
    assert dec.tokens == 0
    # rows of a wider projection
    dec.fill_prefix(torch.ones(4, 1024, **bf)[:, 512:])
    torch.cuda.synchronize()
    assert (dec.cache[:4] == 1).all()


def test_pipeline_prefix_decode_norm_weights_of_any_layout(lib):
    """Norm weights that are a column of a packed matrix, or begin off a 16-byte border, give the
    rows that their contiguous copy gives."""
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    g = torch.Generator(device="cuda").manual_seed(3)
    packed = (1 + 0.1 * torch.randn(512, 8, generator=g, device="cuda")).to(torch.bfloat16)
    flat = packed.reshape(-1)
    x = torch.randn(5, 512, generator=g, device="cuda").to(torch.bfloat16)
    for w in [packed[:, 0], packed[:, 3], flat[5:517], flat[1:1537:3], packed[:, 2].float()]:
        got, want = (PrefixDecode(1, 16, 4, 5, norm_w=v) for v in (w, w.contiguous().clone()))
        for dec in (got, want):
            dec.fill_prefix(x)
        torch.cuda.synchronize()
        assert torch.equal(got.cache.view(torch.uint8), want.cache.view(torch.uint8))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("name", ["dsa_latent_append_paged", "dsa_prefix_mla_decode_paged"])
def test_pipeline_prefix_decode_after_a_call_that_was_refused(lib, monkeypatch, name, graph):
    """A step whose call fails is not taken: the object's lengths stay, and the next step gives
    what it gives on an object that never failed. With a graph the refusal comes at the
    captured call, the second of the step."""
    from sparse_attention_indexer_head_b200 import pipeline
    rng = np.random.default_rng(9)
    cs = torch.from_numpy(cos_sin_table(32))
    x = to_bf16(bf16_round(rng.standard_normal((7, 576))))
    steps = [(to_bf16(bf16_round(rng.standard_normal((2, 576)))), to_bf16(bf16_round(rng.standard_normal((2, 16, 576)))))
             for _ in range(3)]
    made = [pipeline.PrefixDecode(2, 16, 3, 7, norm_w=None, cos_sin=cs, graph=graph) for _ in range(2)]
    for dec in made:
        dec.fill_prefix(x)
    call, count = getattr(pipeline.B, name), [0]

    def refuse(*a, **kw):
        count[0] += 1
        if count[0] > int(graph):
            raise lib.DsaError(name, lib.DSA_ERR_UNSUPPORTED, "refused")
        call(*a, **kw)

    with monkeypatch.context() as m:
        m.setattr(pipeline.B, name, refuse)
        with pytest.raises(lib.DsaError):
            made[0].step(*steps[0])
    assert made[0].tokens == 0 and made[0].seq_len.tolist() == [7, 7] and made[0].q_pos.tolist() == [6, 6]
    for s in steps:
        got, want = [dec.step(*s).clone() for dec in made]
        assert torch.equal(got, want)
    assert lib.dsa_device_status(reset=True) == 0
    for dec in made:
        assert dec.tokens == 3 and dec.seq_len.tolist() == [10, 10]
    assert torch.equal(made[0].cache, made[1].cache)


def test_pipeline_prefix_decode_takes_its_own_buffers(lib):
    """Inputs written straight into the object's buffers: the first step of a graph, which makes
    its calls twice, rotates them once."""
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    rng = np.random.default_rng(10)
    cs = torch.from_numpy(cos_sin_table(32))
    eager, graph = [PrefixDecode(2, 16, 2, 5, norm_w=None, cos_sin=cs, graph=g) for g in (False, True)]
    x = to_bf16(bf16_round(rng.standard_normal((5, 576))))
    for dec in (eager, graph):
        dec.fill_prefix(x)
    for _ in range(2):
        kv_new, q = to_bf16(bf16_round(rng.standard_normal((2, 576)))), to_bf16(bf16_round(rng.standard_normal((2, 16, 576))))
        graph.kv_new.copy_(kv_new)
        graph.q.copy_(q)
        want = eager.step(kv_new, q)
        assert torch.equal(graph.step(graph.kv_new, graph.q), want) and torch.equal(graph.q, eager.q)


def test_pipeline_prefix_decode_has_read_pinned_inputs_when_it_returns(lib):
    """Pinned inputs that are refilled at once, while the stream is still busy with earlier work."""
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    rng = np.random.default_rng(11)
    dec, ref = [PrefixDecode(2, 16, 3, 5, norm_w=None) for _ in range(2)]
    x = to_bf16(bf16_round(rng.standard_normal((5, 512))))
    for d in (dec, ref):
        d.fill_prefix(x)
    kv_new, q = [torch.empty(*s, dtype=torch.bfloat16).pin_memory() for s in ((2, 512), (2, 16, 512))]
    want, got = [], []
    for _ in range(3):
        a, b = to_bf16(bf16_round(rng.standard_normal((2, 512)))), to_bf16(bf16_round(rng.standard_normal((2, 16, 512))))
        want.append(ref.step(a, b).clone())
        kv_new.copy_(a)
        q.copy_(b)
        torch.cuda._sleep(20_000_000)              # 10 ms
        got.append(dec.step(kv_new, q).clone())
        kv_new.fill_(9.0)
        q.fill_(9.0)
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(dec.cache, ref.cache)


@pytest.mark.parametrize("handle", [False, True])
def test_pipeline_prefix_decode_filled_on_another_stream(lib, handle):
    """The fill on a side stream runs behind what the current stream still has to do (the cache's
    zeros, the rows themselves), and the step behind the fill."""
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    rng = np.random.default_rng(12)
    x = to_bf16(bf16_round(rng.standard_normal((300, 512))))
    row, q = to_bf16(bf16_round(rng.standard_normal((1, 512)))), to_bf16(bf16_round(rng.standard_normal((1, 16, 512))))
    ref = PrefixDecode(1, 16, 4, 300, norm_w=None)
    ref.fill_prefix(x)
    want = ref.step(row, q)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    rows = torch.zeros_like(x)
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                  # 10 ms
    dec = PrefixDecode(1, 16, 4, 300, norm_w=None)
    rows.copy_(x)
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)               # the step below must not overtake the fill
    dec.fill_prefix(rows, stream=s.cuda_stream if handle else s)
    got = dec.step(row, q)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(dec.cache, ref.cache)


def test_pipeline_prefix_decode_keeps_its_device(lib):
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    dec = PrefixDecode(1, 16, 4, 4, norm_w=None)
    assert dec.device == dec.cache.device == torch.device("cuda", torch.cuda.current_device())


@pytest.mark.parametrize("graph", [False, True])
def test_pipeline_prefix_decode_keeps_no_autograd_history(lib, graph):
    """Inputs that come out of layers with gradients on: the object's buffers hold none of it."""
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    bf = dict(dtype=torch.bfloat16, device="cuda")
    dec, ref = [PrefixDecode(2, 16, 3, 4, norm_w=torch.nn.Parameter(torch.ones(512, **bf)), graph=graph) for _ in range(2)]
    x, kv_new, q = torch.randn(4, 512, **bf), torch.randn(2, 512, **bf), torch.randn(2, 16, 512, **bf)
    scale = torch.nn.Parameter(torch.ones((), **bf))
    dec.fill_prefix(x * scale)
    ref.fill_prefix(x)
    for _ in range(2):
        got, want = dec.step(kv_new * scale, q * scale), ref.step(kv_new, q)
        assert torch.equal(got, want) and not got.requires_grad
    assert not any(t.requires_grad for t in (dec.kv_new, dec.q, dec.out, dec.lse, dec.cache))


def test_pipeline_prefix_decode_fills_on_the_stream_that_it_is_given(lib, monkeypatch):
    """By handle (0: the default stream), by torch's object or by another that has a handle."""
    from types import SimpleNamespace
    from sparse_attention_indexer_head_b200 import pipeline
    dec = pipeline.PrefixDecode(1, 16, 4, 4, norm_w=None)
    x = torch.ones(4, 512, dtype=torch.bfloat16, device="cuda")
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    call, seen = pipeline.B.dsa_latent_append_paged, []

    def note(*a, stream):
        seen.append(stream.cuda_stream)
        call(*a, stream=stream)

    monkeypatch.setattr(pipeline.B, "dsa_latent_append_paged", note)
    for given in (None, 0, s, s.cuda_stream, SimpleNamespace(cuda_stream=s.cuda_stream), t):
        with torch.cuda.stream(t):
            dec.fill_prefix(x, stream=given)
    dec.fill_prefix(x, stream=0)
    torch.cuda.synchronize()
    assert seen == [t.cuda_stream, 0, s.cuda_stream, s.cuda_stream, s.cuda_stream, t.cuda_stream, 0]
    assert (dec.cache[:4] == 1).all()

"""The paged append and the shared-prefix MLA on the host: refusals before anything is
launched, and the oracle's functions pinned to closed forms."""
import numpy as np
import pytest

import oracle as O
from paged_helpers import cos_sin_table

FAKE = 1 << 20          # a 16-byte aligned non-null address; never dereferenced on these paths


@pytest.fixture(scope="module")
def B():
    from sparse_attention_indexer_head_b200 import build
    build.build()
    from sparse_attention_indexer_head_b200 import binding
    return binding


def _append(api, fp8=False, **kw):
    a = dict(kv_new=FAKE, stride=576, norm_w=FAKE, eps=1e-6, cos_sin=FAKE, max_pos=64, interleaved=1, tok_req=FAKE,
             tok_pos=FAKE, n=4, kv_lora=512, rope=64, table=FAKE, B=2, max_blocks=4, page=16, kv=FAKE, scale=0.5,
             rows=128, q_rot=FAKE, qt=16 * 64, qh=64, Hm=16, q=FAKE)
    a.update(kw)
    head = [a[k] for k in ("kv_new", "stride", "norm_w", "eps", "cos_sin", "max_pos", "interleaved", "tok_req", "tok_pos",
                           "n", "kv_lora", "rope", "table", "B", "max_blocks", "page", "kv")]
    tail = [a[k] for k in ("rows", "q_rot", "qt", "qh", "Hm", "q")]
    if fp8:
        return api.lib.dsa_latent_append_paged_fp8(*head, a["scale"], *tail, None)
    return api.lib.dsa_latent_append_paged(*head, *tail, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,status", [
    (dict(n=-1), 1), (dict(B=-1), 1), (dict(page=0), 1), (dict(max_blocks=-1), 1), (dict(rows=-1), 1),
    (dict(max_pos=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(stride=568), 1),
    (dict(interleaved=2), 1), (dict(kv_new=None), 1), (dict(tok_req=None), 1), (dict(tok_pos=None), 1),
    (dict(table=None), 1), (dict(kv=None), 1), (dict(cos_sin=None), 1), (dict(q=None), 1), (dict(q_rot=None), 1),
    (dict(rope=0, stride=512), 1),                       # heads without a rotation
    (dict(Hm=0), 1), (dict(qh=56), 1), (dict(qt=15 * 64), 1),
    (dict(kv_lora=576), 2), (dict(rope=32), 2), (dict(rope=128, stride=640), 2),
    (dict(Hm=144, qt=144 * 64), 2),
    (dict(kv_new=FAKE + 8), 3), (dict(stride=580), 3), (dict(norm_w=FAKE + 2), 3), (dict(cos_sin=FAKE + 4), 3),
    (dict(tok_req=FAKE + 2), 3), (dict(tok_pos=FAKE + 1), 3), (dict(table=FAKE + 2), 3), (dict(kv=FAKE + 8), 3),
    (dict(q_rot=FAKE + 8), 3), (dict(q=FAKE + 4), 3), (dict(qh=68, qt=16 * 68), 3), (dict(qt=16 * 64 + 4), 3),
])
def test_append_refusals(B, bad, status, fp8):
    assert _append(B, fp8, **bad) == status


def test_append_scale_and_empty_calls(B):
    for scale in (0.0, -1.0, float("inf"), float("nan"), 1e-39):     # 1 / 1e-39 is no fp32 number
        assert _append(B, True, scale=scale) == B.DSA_ERR_INVALID_ARG
    none = dict(kv_new=None, tok_req=None, tok_pos=None, table=None, kv=None, cos_sin=None)
    assert _append(B, n=0, **none) == B.DSA_OK
    assert _append(B, B=0, **none) == B.DSA_OK
    with pytest.raises(B.DsaError):
        B.dsa_latent_append_paged(None, 576, None, 1e-6, None, 0, 1, None, None, 1, 512, 64, None, 1, 1, 0, None, 1, stream=0)


def _mla(api, fp8=False, **kw):
    a = dict(q=FAKE, kv=FAKE, scale=0.5, rows=64, prefix=FAKE, pb=2, plen=FAKE, table=FAKE, mb=4, page=16, seq=FAKE,
             q_req=FAKE, q_pos=FAKE, Q=2, B=2, Hm=32, kv_lora=512, rope=64, sm=0.05, out=FAKE, lse=FAKE, ws=FAKE,
             ws_bytes=1 << 40)
    a.update(kw)
    head = [a["q"], a["kv"]] + ([a["scale"]] if fp8 else [])
    rest = [a[k] for k in ("rows", "prefix", "pb", "plen", "table", "mb", "page", "seq", "q_req", "q_pos", "Q", "B", "Hm",
                           "kv_lora", "rope", "sm", "out", "lse", "ws", "ws_bytes")]
    fn = api.lib.dsa_prefix_mla_decode_paged_fp8 if fp8 else api.lib.dsa_prefix_mla_decode_paged
    return fn(*head, *rest, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad,status", [
    (dict(Q=-1), 1), (dict(B=-1), 1), (dict(Hm=0), 1), (dict(page=0), 1), (dict(mb=-1), 1), (dict(pb=-1), 1),
    (dict(rows=-1), 1), (dict(rope=-1), 1), (dict(sm=float("nan")), 1), (dict(sm=float("inf")), 1), (dict(q=None), 1),
    (dict(kv=None), 1), (dict(prefix=None), 1), (dict(plen=None), 1), (dict(table=None), 1), (dict(seq=None), 1),
    (dict(q_req=None), 1), (dict(q_pos=None), 1), (dict(out=None), 1),
    (dict(kv_lora=576), 2), (dict(rope=32), 2), (dict(Hm=24), 2), (dict(Hm=144), 2), (dict(Q=65536), 2),
    (dict(rows=1 << 31), 2),
    (dict(q=FAKE + 8), 3), (dict(kv=FAKE + 8), 3), (dict(prefix=FAKE + 2), 3), (dict(plen=FAKE + 2), 3),
    (dict(table=FAKE + 2), 3), (dict(seq=FAKE + 2), 3), (dict(q_req=FAKE + 2), 3), (dict(q_pos=FAKE + 2), 3),
    (dict(out=FAKE + 8), 3), (dict(lse=FAKE + 2), 3), (dict(ws=FAKE + 8), 3),
    (dict(ws=None), 4), (dict(ws_bytes=0), 4),
])
def test_prefix_mla_refusals(B, bad, status, fp8):
    assert _mla(B, fp8, **bad) == status


def test_prefix_mla_scale_empty_call_and_workspace(B):
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert _mla(B, True, scale=scale) == B.DSA_ERR_INVALID_ARG
    assert _mla(B, True, scale=1e30, sm=-1e30) == B.DSA_ERR_INVALID_ARG     # the logits' scale overflows
    assert _mla(B, sm=3e38) == B.DSA_ERR_INVALID_ARG                        # with its log2(e) too
    assert _mla(B, Q=0, q=None, q_req=None, out=None, ws=None) == B.DSA_OK
    assert B.dsa_prefix_mla_workspace_size(0, 64) == 0
    for Q, hm in [(1, 16), (64, 128), (65535, 128)]:
        need = B.dsa_prefix_mla_workspace_size(Q, hm)
        assert 0 < need < 64 << 20                     # it does not grow with the batch
        assert _mla(B, Q=Q, Hm=hm, ws_bytes=need - 1) == B.DSA_ERR_WORKSPACE


def test_oracle_rotation_is_a_complex_product():
    rng = np.random.default_rng(0)
    x, cs = rng.standard_normal((3, 64)), cos_sin_table(50)
    c, s = cs[41, :32].astype(float), cs[41, 32:].astype(float)
    turn = c + 1j * s
    y = O.rotate(x, c, s, True)
    np.testing.assert_allclose(y[:, 0::2] + 1j * y[:, 1::2], (x[:, 0::2] + 1j * x[:, 1::2]) * turn, rtol=1e-14, atol=1e-14)
    y = O.rotate(x, c, s, False)
    np.testing.assert_allclose(y[:, :32] + 1j * y[:, 32:], (x[:, :32] + 1j * x[:, 32:]) * turn, rtol=1e-14, atol=1e-14)


def test_oracle_append_places_and_normalises():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 576))
    table = np.array([[2, -1], [0, 1]])
    rows, heads = O.latent_append(x, np.ones(512), 0.0, cos_sin_table(8), True, [0, 1, 0], [1, 5, 4], table, 4, 12,
                                  np.ones((3, 2, 64)))
    assert sorted(rows) == [5, 9] and sorted(heads) == [0, 1, 2]       # token 2's page is missing, its heads turn
    for r in rows.values():
        assert abs((r[:512] ** 2).mean() - 1) < 1e-12
        # a rotation keeps lengths
    assert abs((rows[9][512:] ** 2).sum() - (x[0, 512:] ** 2).sum()) < 1e-5
    np.testing.assert_allclose(rows[9][:512] / rows[9][0], x[0, :512] / x[0, 0], rtol=1e-12)


def test_oracle_prefix_mla_closed_forms():
    kv = np.zeros((16, 512))
    kv[:, 0] = np.arange(16)
    q = np.zeros((3, 1, 512))
    # equal logits: the mean of the values seen; prefix pages 3, own pages 1 and 2
    out, lse, mag, _, seen = O.prefix_mla(q, kv, [3], 3, [[0, 1], [-1, 2]], 4, [6, 7], [0, 1, 5], [9, 5, 0], 1.0)
    # request 0: tokens 0..2 in page 3, token 3 in its own page 0, tokens 4, 5 in page 1
    assert seen.tolist() == [6, 5, 0]
    assert out[0, 0, 0] == pytest.approx((12 + 13 + 14 + 3 + 4 + 5) / 6)
    # request 1 has no page for token 3; tokens 4, 5 in page 2
    assert out[1, 0, 0] == pytest.approx((12 + 13 + 14 + 8 + 9) / 5)
    assert lse[0, 0] == pytest.approx(np.log(6)) and np.isneginf(lse[2]).all() and (out[2] == 0).all()
    # one token: its value, whatever the logits
    out, lse, *_ = O.prefix_mla(np.ones((1, 1, 512)), kv, [], 0, [[2]], 4, [1], [0], [0], 0.5)
    assert out[0, 0, 0] == 8 and lse[0, 0] == pytest.approx(4.0)


def test_fast_calls_convert_like_the_declarations(B):
    """The extension module's calls against the same refusals through ctypes."""
    import torch
    call, t = B._call, torch.zeros(64, dtype=torch.float32)
    # None, an address and a tensor are pointers; the status comes back as it is
    assert call.dsa_head_gate(None, None, None, 4, 4096, 16, None) == B.DSA_ERR_INVALID_ARG
    assert call.dsa_head_gate(FAKE + 4, FAKE, t, 4, 4096, 16, 0) == B.DSA_ERR_ALIGNMENT
    assert call.dsa_head_gate(t, t, t, 0, 4096, 16, None) == B.DSA_OK
    args = [FAKE] * 4 + [2, 128, 9, 8, FAKE, FAKE, FAKE, 1e-5] + [FAKE] * 4 + [None]
    assert call.dsa_kpool_compress(*args) == B.lib.dsa_kpool_compress(*args) == B.DSA_ERR_UNSUPPORTED
    args[11] = float("nan")
    assert call.dsa_kpool_compress(*args) == B.lib.dsa_kpool_compress(*args)
    assert call.dsa_head_gate(FAKE, FAKE, FAKE, np.int64(4), np.int32(4094), 16, None) == B.DSA_ERR_UNSUPPORTED
    with pytest.raises(TypeError):
        call.dsa_head_gate(None, None, None, 4, 4096, 16)
    with pytest.raises(TypeError):
        call.dsa_head_gate(None, None, None, 4.5, 4096, 16, None)
    with pytest.raises(AttributeError):
        call.dsa_head_gate("text", None, None, 4, 4096, 16, None)
    with pytest.raises(OverflowError):
        call.dsa_head_gate(None, None, None, 1 << 31, 4096, 16, None)
    with pytest.raises(OverflowError):
        call.dsa_sparse_mla_decode(*[FAKE] * 2, 64, *[FAKE] * 3, 1, 1, 16, 48, 512, 0, 0.1, FAKE, None, FAKE, -1, None)


def test_every_launching_entry_point_has_a_fast_call(B):
    queries = {"dsa_status_string", "dsa_abi_version", "dsa_device_status", "dsa_head_gate_supported",
               "dsa_sparse_mla_workspace_size", "dsa_sparse_mla_launch_count", "dsa_noalloc_scratch_bytes",
               "dsa_prefix_mla_workspace_size"}
    assert {n for n in dir(B._call) if n.startswith("dsa_")} == set(B.EXPORTS) - queries


def _refused(**kw):
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    a = dict(requests=2, heads=16, max_own=8, prefix_len=4, norm_w=None)
    a.update(kw)
    with pytest.raises(ValueError):
        PrefixDecode(a.pop("requests"), a.pop("heads"), a.pop("max_own"), a.pop("prefix_len"), **a)


def test_prefix_decode_refuses_norm_weights_of_another_shape(B):
    import torch
    for shape in [(256,), (511,), (513,), (1, 512), (512, 1), ()]:
        _refused(norm_w=torch.ones(shape), device="cpu")
        _refused(norm_w=torch.ones(shape, dtype=torch.bfloat16), device="cpu")


def test_operands_are_dense_and_aligned(B):
    import torch
    from sparse_attention_indexer_head_b200.pipeline import _operand
    wide = torch.arange(2048, dtype=torch.float32).to(torch.bfloat16)
    for x in [wide[::2], wide[:1024:2], wide.view(2, 1024).t()[:512, 1], wide[3:515], wide[1:].view(-1)[:512], wide[:512]]:
        y = _operand(x, torch.device("cpu"), torch.bfloat16)
        assert torch.equal(x, y) and y.is_contiguous() and y.data_ptr() % 16 == 0
    x = wide[8:520]                                       # usable as it lies: no copy
    assert _operand(x, torch.device("cpu"), torch.bfloat16).data_ptr() == x.data_ptr()


@pytest.mark.parametrize("kw", [
    dict(heads=0), dict(heads=24), dict(heads=144), dict(sm_scale=float("nan")), dict(sm_scale=3e38), dict(eps=-1.0),
    dict(eps=float("inf")), dict(fp8=True, kv_scale=0.0), dict(fp8=True, kv_scale=1e-39), dict(fp8=True, kv_scale=float("inf")),
    dict(fp8=True, kv_scale=1e30, sm_scale=1e30), dict(rope=32), dict(rope=128), dict(max_own=1 << 31, requests=1),
])
def test_prefix_decode_refuses_at_once_what_its_calls_refuse(B, kw):
    import torch
    from sparse_attention_indexer_head_b200.pipeline import PrefixDecode
    a = dict(requests=2, heads=16, max_own=8, prefix_len=4, norm_w=None)
    a.update(kw)
    if "rope" in a:
        a["cos_sin"] = torch.zeros(64, a.pop("rope"))
    with pytest.raises(B.DsaError) as e:
        PrefixDecode(a.pop("requests"), a.pop("heads"), a.pop("max_own"), a.pop("prefix_len"), **a)
    assert e.value.status in (B.DSA_ERR_INVALID_ARG, B.DSA_ERR_UNSUPPORTED)


def test_prefix_decode_refuses_sizes(B):
    import torch
    for kw in [dict(requests=-1), dict(max_own=-1), dict(prefix_len=-1), dict(page=0), dict(page=-16), dict(requests=65536),
               dict(cos_sin=torch.zeros(11, 64)), dict(cos_sin=torch.zeros(64)), dict(cos_sin=torch.zeros(64, 32, 2))]:
        _refused(**kw)


def test_prefix_decode_is_of_one_cuda_device(B, monkeypatch):
    """A device without a number is the current one at the time, and stays it."""
    import torch
    from sparse_attention_indexer_head_b200 import pipeline
    _refused(device="cpu")
    _refused(device="meta")
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    seen = []

    def stop(x, device, dtype):
        seen.append(device)
        raise KeyError                                     # before anything is allocated

    monkeypatch.setattr(pipeline, "_operand", stop)
    for device in ("cuda", "cuda:1"):
        with pytest.raises(KeyError):
            pipeline.PrefixDecode(1, 16, 4, 4, norm_w=torch.ones(512), device=device)
    assert seen == [torch.device("cuda", 3), torch.device("cuda", 1)]


@pytest.mark.parametrize("fp8", [False, True])
def test_prefix_mla_tables_too_long_for_the_plan(B, fp8):
    """Work beyond the plan's counts (32 row tiles' units of 32 tokens in 32 bits, a CTA's in 31) is
    refused; a call that is not goes on to the workspace check, never to a launch."""
    def status(tokens, Q, Hm, at="mb"):
        page = next(p for p in (1 << 20, 1 << 16, 1) if tokens % p == 0)
        return _mla(B, fp8, **{at: tokens // page}, page=page, Q=Q, B=Q, Hm=Hm, ws=None)

    for Q, Hm, most in [(128, 16, (1 << 30) - 128), (65535, 64, 1 << 26), (65535, 128, 1 << 26), (65535, 16, 1 << 26),
                        (96, 32, (1 << 31) - 1), (4000, 64, (1 << 31) - 1), (1, 16, (1 << 31) - 1), (124, 16, 1 << 30)]:
        for at in ("mb", "pb"):
            assert status(most, Q, Hm, at) == B.DSA_ERR_WORKSPACE, (Q, Hm, most)
    for Q, Hm, tokens in [(128, 16, 1 << 30), (128, 16, (1 << 31) - 1), (5000, 64, (1 << 31) - 1), (65535, 128, 1 << 28),
                          (65535, 16, 1 << 29)]:
        for at in ("mb", "pb"):
            assert status(tokens, Q, Hm, at) == B.DSA_ERR_UNSUPPORTED, (Q, Hm, tokens)
    # what the bound stands for: tiles of qpt queries, each over the whole of its table
    for Q, Hm, tokens in [(128, 16, (1 << 30) - 128), (65535, 128, 1 << 26), (65535, 16, 1 << 26), (96, 32, (1 << 31) - 65)]:
        qpt = max(1, 64 // Hm) if Hm < 64 else 1
        tiles = -(-Q // qpt) if qpt > 1 else Q * -(-Hm // 64)
        tile = qpt * (tokens // 32 + 1) + 1
        assert min(32, tiles) * tile < 1 << 32 and -(-tiles * tile // 148) < 1 << 31


def test_calls_convert_numbers_as_before(B):
    """Row counts and workspace sizes given as floats, scales as anything that float() takes: calls
    that launch nothing (no query, no request) get through, refusals keep their status."""
    for rows, size in [(64, 4096), (64.0, 4096.0), (np.float64(64), np.int64(4096)), ("64", "4096")]:
        for sm in (0.1, "0.1", np.float32(0.1)):
            B.dsa_sparse_mla_decode(FAKE, FAKE, rows, FAKE, FAKE, FAKE, 0, 1, 16, 48, 512, 0, sm, FAKE, None, FAKE, size, 0)
            B.dsa_sparse_mla_decode_noalloc(FAKE, FAKE, rows, FAKE, FAKE, FAKE, 0, 1, 16, 48, 512, 0, sm, FAKE, None, 0)
    for sm in (0.1, "0.1", np.float32(0.1)):
        B.dsa_sparse_mla_decode_paged(FAKE, FAKE, 64, FAKE, 2, 16, FAKE, FAKE, FAKE, 0, 1, 16, 48, 512, 0, sm, FAKE, None, FAKE, 0, 0)
        B.dsa_sparse_mla_decode_paged_fp8(FAKE, FAKE, sm, 64, FAKE, 2, 16, FAKE, FAKE, FAKE, 0, 1, 16, 48, 512, 0, sm, FAKE, None,
                                          FAKE, 0, 0)
    for eps in ("nan", "-1", -1):
        with pytest.raises(B.DsaError):
            B.dsa_kpool_compress(FAKE, FAKE, FAKE, FAKE, 2, 128, 4, 8, FAKE, FAKE, FAKE, eps, FAKE, FAKE, FAKE, FAKE, 0)
        with pytest.raises(B.DsaError):
            B.dsa_kpool_compress_tokens(FAKE, FAKE, FAKE, FAKE, 2, 128, 4, 8, FAKE, FAKE, FAKE, eps, FAKE, FAKE, FAKE, FAKE, FAKE,
                                        FAKE, 0)


def test_extension_module_is_of_this_interpreter(B):
    """Another Python version's module has another name, so that it is not loaded."""
    import sysconfig
    from sparse_attention_indexer_head_b200 import build
    assert build.CALL.endswith(sysconfig.get_config_var("EXT_SUFFIX"))
    assert B._call.__spec__.origin == build.CALL

"""Shared pieces of the latent append and shared-prefix MLA tests: random paged batches and
the tolerances, each counted from the roundings of the computation."""
import numpy as np
import torch

import oracle as O
from sparse_attention_indexer_head_b200 import workloads as W

HALF_BF16 = 2.0 ** -8            # half a step of bf16, relative
HALF_E4M3 = 2.0 ** -4            # half a step of E4M3, relative, above its subnormals
SUB_E4M3 = 2.0 ** -10            # half a step of its subnormals


def bf16_round(x):
    return W.bf16_bits_to_f32(W.f32_to_bf16_bits(np.asarray(x, np.float32)))


def to_bf16(x):
    """Real numbers to a device bf16 tensor (NaN and infinities kept)."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).cuda().to(torch.bfloat16)


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def scatter_pages(counts, page, rng, spare=2):
    """Scattered pages for sequences of `counts` tokens: ([n, most] table with -1, pool pages)."""
    need = [-(-int(c) // page) for c in counts]
    order = rng.permutation(sum(need) + spare)
    table = np.full((len(counts), max(1, max(need, default=1))), -1, np.int32)
    at = 0
    for i, k in enumerate(need):
        table[i, :k] = order[at:at + k]
        at += k
    return table, len(order)


def cos_sin_table(n, rope=64, base=10000.0):
    a = np.arange(n)[:, None] * base ** (-np.arange(rope // 2) * 2.0 / rope)
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)


class Batch:
    """A batch behind a shared prefix: pages, lengths and values, cache rows that no token
    owns hold `fill` (NaN: a read of a wrong row shows)."""

    def __init__(self, seed, own, prefix=0, page=32, hm=16, rope=64, per=1, fp8=False, fill=np.nan,
                 scale=0.25, q_req=None, q_pos=None, drop=(), spread=1.0):
        rng = np.random.default_rng(seed)
        self.own, self.P, self.page, self.hm, self.rope, self.fp8 = list(own), prefix, page, hm, rope, fp8
        self.scale, self.width, self.B = scale, 512 + rope, len(own)
        self.sm_scale = float(np.float32(1 / np.sqrt(self.width)))
        whole = prefix // page * page
        both, pages = scatter_pages([prefix] + [prefix - whole + n for n in own], page, rng)
        self.prefix_table = both[0, :max(1, -(-prefix // page))]
        self.table = np.concatenate([np.full((self.B, whole // page), -1, np.int32), both[1:]], 1)
        for b, pi in drop:
            self.table[b, pi] = -1
        self.seq_len = np.asarray([prefix + n for n in own], np.int32)
        self.q_req = np.repeat(np.arange(self.B), per) if q_req is None else np.asarray(q_req)
        if q_pos is None:
            q_pos = (self.seq_len[:, None] + np.arange(per) - per).reshape(-1)
        self.q_pos = np.asarray(q_pos)
        self.Q = len(self.q_req)
        rows = pages * page
        values = bf16_round(rng.standard_normal((rows, self.width)) * spread)
        owned = np.zeros(rows, bool)
        for t in range(prefix):
            owned[O.paged_row(self.prefix_table, page, t, rows)] = True
        for b in range(self.B):
            for t in range(prefix, int(self.seq_len[b])):
                r = O.paged_row(self.table[b], page, t, rows)
                if r >= 0:
                    owned[r] = True
        if fp8:
            codes = rng.integers(0, 256, (rows, self.width)).astype(np.uint8)
            codes[(codes & 0x7F) >= 0x60] ^= 0x40          # values up to 3.75, no NaN
            codes[~owned] = 0x7F if np.isnan(fill) else 0
            self.codes = codes
            values = O.e4m3_to_f64(codes) * np.float32(scale)
        else:
            values[~owned] = fill
        self.values, self.owned, self.rows = values, owned, rows
        self.q = bf16_round(rng.standard_normal((self.Q, hm, self.width)))

    def device(self):
        cache = torch.from_numpy(self.codes).cuda() if self.fp8 else to_bf16(self.values)
        return dict(q=to_bf16(self.q), cache=cache, prefix_table=i32(self.prefix_table),
                    prefix_len=i32([self.P]), table=i32(self.table), seq_len=i32(self.seq_len),
                    q_req=i32(self.q_req), q_pos=i32(self.q_pos))

    def buffers(self, lib):
        ws = torch.empty(max(16, lib.dsa_prefix_mla_workspace_size(self.Q, self.hm)), dtype=torch.uint8,
                         device="cuda")
        return dict(out=torch.full((self.Q, self.hm, 512), float("nan"), dtype=torch.bfloat16, device="cuda"),
                    lse=torch.full((self.Q, self.hm), float("nan"), device="cuda"), ws=ws.fill_(0xFF))

    def call(self, lib, d, o, stream=None):
        args = (d["prefix_table"], len(self.prefix_table), d["prefix_len"], d["table"], self.table.shape[1],
                self.page, d["seq_len"], d["q_req"], d["q_pos"], self.Q, self.B, self.hm, 512, self.rope,
                self.sm_scale, o["out"], o["lse"], o["ws"], o["ws"].numel(), stream)
        if self.fp8:
            lib.dsa_prefix_mla_decode_paged_fp8(d["q"], d["cache"], float(np.float32(self.scale)), self.rows, *args)
        else:
            lib.dsa_prefix_mla_decode_paged(d["q"], d["cache"], self.rows, *args)

    def oracle(self):
        return O.prefix_mla(self.q, self.values, self.prefix_table, self.P, self.table, self.page,
                            self.seq_len, self.q_req, self.q_pos, self.sm_scale)

    def run_and_check(self, lib):
        d, o = self.device(), self.buffers(lib)
        self.call(lib, d, o)
        torch.cuda.synchronize()
        self.check(lib, o)
        return d, o

    def check(self, lib, o, want=None):
        assert lib.dsa_device_status(reset=True) == 0
        assert_attention_close(o["out"].float().cpu().numpy(), o["lse"].cpu().numpy(),
                               self.oracle() if want is None else want, self.width)


def assert_attention_close(out, lse, want, width):
    """Shared-prefix MLA against the oracle in 64 bits.

    Roundings, T tokens and a logit z of `width` terms whose absolute values add up to Z:
      logits: products exact in fp32 and at most width + 8 additions (a truncating
        accumulator: 2^-23 each), a scale of two roundings and the exponential's argument,
        |z| <= Z: dz <= (width + 12) 2^-23 Z; the exponential itself 2^-21;
      weights: bf16 in the product with the values: half a step, HALF_BF16;
      sums: T + 8 additions of fp32 (2^-23 each), of weights in the denominator and of
        weighted values, merges of parts included;
      output: half a step of bf16 of the result.
    With A the softmax-weighted mean of |v|: |out - ref| <= HALF_BF16 |ref| + A (HALF_BF16 +
    2 (dz + 2^-21) + 2 (T + 8) 2^-23), times 1 + 2^-6 for products of these; and
    |lse - ref| <= dz + 2^-21 + (T + 8) 2^-23 + 2^-22 |ref|.
    """
    ref, rlse, mag, terms, seen = want
    none = np.isneginf(rlse)
    assert (np.isneginf(lse) == none).all(), "rows without a token: lse = -inf there and only there"
    assert (out[none] == 0).all(), "rows without a token: out = 0"
    dz = (width + 12) * 2.0 ** -23 * terms + 2.0 ** -21
    sums = (seen[:, None] + 8) * 2.0 ** -23
    tol = (HALF_BF16 * np.abs(ref) + mag * (HALF_BF16 + 2 * dz + 2 * sums)[..., None]) * (1 + 2.0 ** -6)
    err = np.abs(out - ref)
    assert (err <= tol).all(), f"{(~(err <= tol)).sum()} outputs outside, worst {np.nanmax(err - tol):.3g} over"
    lerr = np.abs(lse[~none] - rlse[~none])
    ltol = (dz + sums + 2.0 ** -22 * np.abs(np.where(none, 0.0, rlse)))[~none]
    assert (lerr <= ltol).all(), f"lse off by {lerr.max():.3g}"

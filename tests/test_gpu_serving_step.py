"""A serving loop through the paged cache, the calls as a server makes them: reserve pages for a
prompt, rotate and store its keys (rope_append), attend it (fwd_varlen_paged), fork the prompt into
several answers, extend them by chunks and by single tokens (decode_paged), drop some, compact the
pool and go on.  Every output is compared with the attention of the sequence's own tokens, kept
beside the cache, in 64 bits."""
import os
import subprocess
import sys

import pytest
import torch

from exact_io_aware_81_b200 import ops
from oracle import serving
from parity import compare

pytestmark = pytest.mark.gpu

DEV = "cuda"
HERE = os.path.dirname(os.path.abspath(__file__))


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).to(DEV)


class Server:
    def __init__(self, S, Hq, Hkv, d, ps, max_pages, num_pages, A, inter, fp8=False, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.S, self.Hq, self.Hkv, self.d, self.ps, self.A, self.inter, self.fp8 = S, Hq, Hkv, d, ps, A, inter, fp8
        self.table = torch.full((S, max_pages), -1, dtype=torch.int32, device=DEV)
        self.lens, self.ref = i32([0] * S), i32([0] * num_pages)
        shape = (num_pages, Hkv, ps, d)
        if fp8:
            self.kp, self.vp = (torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))  # NaN
            self.ks, self.vs = (torch.rand(Hkv, generator=self.g) * 0.01 + 0.005 for _ in range(2))
        else:
            self.kp, self.vp = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.inv = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float()
        self.axes = (torch.arange(d // 2) * A // (d // 2)).to(torch.int32)
        self.k = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(S)]  # what the cache should hold
        self.v = [torch.zeros(0, Hkv, d, dtype=torch.float64) for _ in range(S)]

    def pages_ok(self):
        lens = self.lens.tolist()
        assert lens == [len(x) for x in self.k]
        held = torch.zeros(len(self.ref), dtype=torch.int32)
        for s, n in enumerate(lens):
            for j in range(-(-n // self.ps)):
                held[int(self.table[s, j])] += 1
        assert torch.equal(self.ref.cpu(), held)

    def step(self, new, how):
        """new[s] tokens for slot s; `how`: fwd_varlen_paged of all, or decode (one token each)."""
        add = [new.get(s, 0) for s in range(self.S)]
        copies = ops.pages_reserve(self.table, self.lens, self.ref, i32(add), self.ps)
        ops.pages_copy(self.kp, self.vp, copies)
        slots = [s for s in range(self.S) if add[s]]
        n = [add[s] for s in slots]
        T = sum(n)
        cu = torch.tensor([0] + n).cumsum(0)
        q, k, v = (torch.randn(T, h, self.d, generator=self.g).to(torch.bfloat16) for h in (self.Hq, self.Hkv, self.Hkv))
        pos = torch.randint(0, 5000, (self.A, T), generator=self.g, dtype=torch.int32)
        table, lens = self.table[slots].contiguous(), self.lens[slots].contiguous()
        kw = dict(k_scale=self.ks.to(DEV), v_scale=self.vs.to(DEV)) if self.fp8 else {}
        qo = ops.rope_append(q.to(DEV), k.to(DEV), v.to(DEV), pos.to(DEV), self.inv.to(DEV), self.kp, self.vp, table,
                             i32(cu), lens, axes=self.axes.to(DEV), interleaved=self.inter, **kw)
        # the rounded values that the cache holds, for the comparison
        rows = serving.token_rows(table.cpu().numpy(), cu.tolist(), lens.tolist(), self.ps, T)
        rk = serving.rope(k, pos, self.inv, self.axes, self.inter)
        for i, s in enumerate(slots):
            t = range(int(cu[i]), int(cu[i + 1]))
            got_k = torch.stack([self.kp[rows[x][0], :, rows[x][1]].cpu() for x in t])
            got_v = torch.stack([self.vp[rows[x][0], :, rows[x][1]].cpu() for x in t])
            if self.fp8:
                got_k = got_k.view(torch.float8_e4m3fn).double() * self.ks.double()[:, None]
                got_v = got_v.view(torch.float8_e4m3fn).double() * self.vs.double()[:, None]
                # half a step of E4M3 (2^-4 relative, 2^-10 among subnormals) of the saturated quotient;
                # the 32-bit rotation's and scaling's errors are far below the last term
                sc = self.ks.double()[:, None]
                ref = rk[t.start:t.stop].clamp(-448 * sc, 448 * sc)
                assert ((got_k - ref).abs() <= 2.0 ** -4 * ref.abs() + 2.0 ** -10 * sc + 1e-5).all()
            else:
                assert ((got_k.double() - rk[t.start:t.stop]).abs() <= 2.0 ** -7 * rk[t.start:t.stop].abs() + 1e-5).all()
                assert torch.equal(got_v, v[t.start:t.stop])
            self.k[s] = torch.cat([self.k[s], got_k.double()])
            self.v[s] = torch.cat([self.v[s], got_v.double()])
        scale = self.d ** -0.5
        if how == "decode":
            assert all(x == 1 for x in n)
            if self.fp8:
                o, lse = ops.decode_paged_fp8(qo, self.kp, self.vp, kw["k_scale"], kw["v_scale"], table, lens)
            else:
                o, lse = ops.decode_paged(qo, self.kp, self.vp, table, lens)
            lse = lse.T
        else:
            o, lse = ops.fwd_varlen_paged(qo, self.kp, self.vp, table, i32(cu), lens, causal=True)
        assert ops.get_error() == ops.FA_OK
        qd = qo.cpu()
        for i, s in enumerate(slots):
            t = slice(int(cu[i]), int(cu[i + 1]))
            ro, rl = serving.attention(qd[t], self.k[s], self.v[s], scale, True)
            compare(o[t], lse[:, t], ro, rl, f"slot {s} {how}")
        self.pages_ok()

    def fork(self, src, dst, lengths=None):
        ops.pages_fork(self.table, self.lens, self.ref, i32(src), i32(dst), self.ps,
                       lengths=i32(lengths) if lengths is not None else None)
        for i, (a, b) in enumerate(zip(src, dst)):
            n = len(self.k[a]) if lengths is None else lengths[i]
            self.k[b], self.v[b] = self.k[a][:n], self.v[a][:n]
        self.pages_ok()

    def drop(self, slots, keep=None):
        ops.pages_free(self.table, self.lens, self.ref, i32(slots), self.ps, keep=i32(keep) if keep else None)
        for i, s in enumerate(slots):
            n = keep[i] if keep else 0
            self.k[s], self.v[s] = self.k[s][:n], self.v[s][:n]
        self.pages_ok()

    def compact(self):
        copies = ops.pages_compact(self.table, self.lens, self.ref, self.ps)
        ops.pages_copy(self.kp, self.vp, copies)
        live = int((self.ref > 0).sum())
        assert (self.ref[live:] == 0).all()
        self.pages_ok()


@pytest.mark.parametrize("Hq,Hkv,d,ps,A,inter", [(8, 2, 128, 16, 3, False), (4, 4, 64, 48, 1, True), (6, 2, 128, 64, 2, False)])
def test_serving(Hq, Hkv, d, ps, A, inter):
    s = Server(7, Hq, Hkv, d, ps, 40, 120, A, inter)
    s.step({0: 170, 1: 33, 2: 1}, "prefill")     # prompts of different lengths at once
    s.fork([0, 0, 1], [3, 4, 5])                 # several answers from one prompt
    s.step({0: 1, 1: 1, 2: 1, 3: 1, 4: 1, 5: 1}, "decode")
    s.step({3: 70, 4: 5, 2: 1, 5: 1}, "prefill") # chunks beside single tokens
    s.drop([0, 5])
    s.drop([3, 4], [180, 171])                   # rejected tokens
    s.compact()
    s.step({1: 1, 2: 1, 3: 1, 4: 1}, "decode")
    s.fork([3], [0], [64])                       # a prefix of another answer
    s.step({0: 20, 6: 90}, "prefill")
    s.step({x: 1 for x in (0, 1, 2, 3, 4, 6)}, "decode")


def test_serving_fp8():
    """The E4M3 cache (no packed prefill over it: its prompts are stored, then decoded)."""
    s = Server(5, 8, 2, 128, 32, 20, 60, 2, False, fp8=True)
    s.step({0: 1, 1: 1}, "decode")
    for _ in range(3):
        s.step({0: 1, 1: 1}, "decode")
    s.fork([0, 1], [2, 3])
    s.step({0: 1, 1: 1, 2: 1, 3: 1}, "decode")
    s.drop([0])
    s.compact()
    s.step({1: 1, 2: 1, 3: 1}, "decode")


def test_bounds_checking_build_finds_nothing():
    """The serving calls' tests through the debug build, whose kernels check every index."""
    lib = os.path.join(os.path.dirname(HERE), "exact_io_aware_81_b200", "libfa_debug.so")
    if os.environ.get("FA_LIBRARY"):
        pytest.skip("already on a chosen build")
    env = dict(os.environ, FA_LIBRARY=lib)
    for name, pick in (("test_gpu_serving_step.py", "serving"), ("test_gpu_rope.py", "append or in_place"),
                       ("test_gpu_varlen.py", "other_keys or paged or fp32 or bad")):
        r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-k", pick, os.path.join(HERE, name)],
                           env=env, cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=600)
        assert r.returncode == 0 and " passed" in r.stdout, r.stdout[-2000:] + r.stderr[-1000:]

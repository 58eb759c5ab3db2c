"""Random paged caches of every type with their float64 values, for the GPU tests."""
import numpy as np
import torch

from oracle import formats, fp4

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


class Paged:
    """A pool of random rows and shuffled tables for sequences of the given lengths.

    k and v: float64 [num_blocks, heads, block, dim], head scales included; the device pools hold the same."""

    def __init__(self, lens, kv, heads, dim, block=16, scaled=True, seed=0, extra=3, max_blocks=None):
        rng = np.random.default_rng(seed + sum(lens) + 17 * heads)
        self.kv, self.heads, self.dim, self.block, self.lens = kv, heads, dim, block, list(lens)
        need = [-(-n // block) for n in lens]
        self.num_blocks = sum(need) + extra
        order = rng.permutation(self.num_blocks)
        width = max(need + [1]) if max_blocks is None else max_blocks
        self.tables = np.full((len(lens), width), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.tables[i, :n] = order[at:at + n]
            at += n
        self.scales = [None, None]
        if kv == "e4m3" or (kv == "fp4" and scaled):
            self.scales = [(0.3 + 1.5 * rng.random(heads)).astype(np.float32) for _ in range(2)]
        self.stored = []
        for _ in range(2):
            x = rng.standard_normal((self.num_blocks, heads, block, dim))
            if kv == "fp4":
                self.stored.append(fp4.pack(*fp4.quantise(x)))
            elif kv == "e4m3":
                self.stored.append(torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
            else:
                self.stored.append(torch.from_numpy(x).to(DT[kv]).view(torch.int16).numpy())
        self.upload()

    def upload(self):
        """The device pools and the values of what `stored` holds now."""
        import paged_kv_cache_160_gb300 as pkv
        dev = [torch.from_numpy(np.ascontiguousarray(s)).cuda() for s in self.stored]
        if self.kv in DT:
            dev = [d.view(DT[self.kv]) for d in dev]
        self.k_cache, self.v_cache = dev
        self.dev_scales = [None if s is None else torch.from_numpy(s).cuda() for s in self.scales]
        make = pkv.cache_desc_fp4 if self.kv == "fp4" else pkv.cache_desc
        self.desc = make(self.k_cache, *self.dev_scales)
        self.dev_tables = torch.from_numpy(self.tables).cuda()
        self.k, self.v = (self.values(s, h) for s, h in zip(self.stored, self.scales))

    def values(self, stored, head_scale=None):
        if self.kv == "fp4":
            x = fp4.values(*fp4.unpack(stored))
        else:
            x = formats.to_f64(stored.view(np.uint8 if self.kv == "e4m3" else np.uint16), self.kv)
        return x if head_scale is None else x * head_scale.astype(np.float64)[:, None, None]

    def rows(self, which, i, n):
        """float64 [n, heads, dim]: positions 0 .. n - 1 of sequence i."""
        pool = self.k if which == "k" else self.v
        j = np.arange(n)
        return pool[self.tables[i, j // self.block], :, j % self.block]

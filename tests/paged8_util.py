"""Problems of the 8-bit cache: pools of codes with NaN wherever no live entry is."""
import numpy as np

from oracle import paged8
from tests.test_gpu_paged import Problem


class Problem8(Problem):
    """Problem's layout; `pools` are what the codes stand for (float64), codes and
    scales the cache itself.  Blocks without a live entry have a scale byte of 255."""

    def __init__(self, seed, dtype, D, Hk, Hq, page, block, q_lens, kv_lens, prefix=0, heads_first=False, pad_rows=0, spread=2):
        import torch
        super().__init__(seed, dtype, D, Hk, Hq, page, q_lens, kv_lens, prefix, heads_first, pad_rows)
        self.block = block
        rng = np.random.default_rng(seed + 1)
        self.codes, self.scales = [], []
        for i in range(2):
            x = self.pools[i].double().cpu().numpy() * 2.0 ** rng.uniform(-spread, spread, self.pools[i].shape[:3])[..., None]
            # (paged8.exponent and quantise for all blocks at once)
            blocks = x.reshape(x.shape[0], page // block, block, Hk, D)
            live = np.isfinite(blocks)
            top = np.abs(np.where(live, blocks, 0)).max(axis=(2, 4))
            e = np.maximum(np.frexp(top)[1] - 8, paged8.LOW[dtype])
            scales = np.where(live.any(axis=(2, 4)), e + 127, 255).astype(np.uint8)
            codes = paged8.quantise(blocks, e[:, :, None, :, None].astype(np.float64), dtype).reshape(x.shape)
            self.codes.append(self._pool(codes, heads_first))
            self.scales.append(torch.from_numpy(scales).cuda())
        self.refresh()

    @staticmethod
    def _pool(codes, heads_first):
        import torch
        t = torch.from_numpy(codes).cuda()
        return t.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else t

    def refresh(self):
        """`pools` from the codes."""
        import torch
        self.pools = [torch.from_numpy(paged8.values(c.cpu().numpy(), s.cpu().numpy())).cuda()
                      for c, s in zip(self.codes, self.scales)]

    def cache(self, sv):
        import torch
        codes = [c.view(torch.float8_e4m3fn) for c in self.codes]
        scales = [s.view(torch.float8_e8m0fnu) for s in self.scales]
        return sv.make_kv_cache8(*codes, *scales, {"bf16": torch.bfloat16, "fp16": torch.float16}[self.dtype])

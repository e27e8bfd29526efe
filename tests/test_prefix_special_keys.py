"""Shared-prefix attention over a visible key with an infinity among its value columns: the definition's NaN, wherever the
key lies and whichever rows share its block."""
import numpy as np
import pytest
import torch

from oracle import cache_ops as C
from test_prefix_attn import BF, F32, Setup


class OneInfinity(Setup):
    """Sequence 0's key at position x has -inf in value column c, where every query is positive: its logit is -inf and
    its probability 0 in every row that sees it, so those rows' column c is 0 times -inf and the rest is as without the key."""

    def __init__(self, x, c, *args, **kw):
        super().__init__(*args, **kw)
        self.x, self.c = x, c
        self.q[..., c] = self.q[..., c].abs() + 0.25
        if self.page:
            at = int(self.prob.block_table[0, x // self.page]) * self.page + x % self.page
        else:
            at = x
        self.kv[at, c] = -float("inf")

    def rows(self):
        for t, q, keys in super().rows():
            sees = t < self.q_lens[0] and len(keys) > self.P + self.x
            yield t, q, np.delete(keys, self.P + self.x, axis=0) if sees else keys

    def check_all(self, out, lse):
        out = out.clone()
        seen = 0
        for t, q, keys in self.rows():
            if t < self.q_lens[0] and self.k_lens[0] - self.q_lens[0] + t >= self.x:
                seen += 1
                assert torch.isnan(out[t, :, self.c]).all(), t
                ro = C.attend(q, keys, self.d_c, self.scale)[0]
                out[t, :, self.c] = torch.from_numpy(ro[:, self.c]).to(out)
        assert seen == min(self.q_lens[0], self.k_lens[0] - self.x)
        self.check(out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("dtype,d_c,d_rope,c", [(BF, 512, 64, 3), (BF, 512, 64, 300), (BF, 512, 0, 511), (BF, 64, 16, 63),
                                                (BF, 272, 48, 260), (F32, 64, 16, 5)])
@pytest.mark.parametrize("q_lens,k_lens,P,x", [
    ([40, 1], [100, 30], 70, 80),       # blocks of several tokens: some see the key, some do not
    ([40, 1], [100, 30], 70, 64),       # at a chunk's start
    ([40, 1], [100, 30], 70, 99),       # seen by the last token alone
    ([3, 1], [100, 30], 0, 20),         # in a chunk that all rows see
    ([2], [65], 4000, 64),              # the only key that a row has in its piece
    ([2, 1, 1], [65, 9, 300], 1, 63),
    ([1], [65], 9001, 64),
])
@pytest.mark.parametrize("h", [1, 16, 128])
def test_infinity_in_a_value_column(q_lens, k_lens, P, x, h, dtype, d_c, d_rope, c, page):
    s = OneInfinity(x, c, q_lens, k_lens, h, d_c, d_rope, P, dtype, page=page, seed=h + x)
    s.check_all(*s.run())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d_c,d_rope", [(BF, 512, 64), (BF, 64, 16), (F32, 64, 16)])
def test_infinity_in_a_piece_without_weight(dtype, d_c, d_rope):
    """One prefix key takes all weight: the piece with the infinity is merged with weight 0, and 0 times its NaN is NaN."""
    s = OneInfinity(40, 9, [1], [41], 1, d_c, d_rope, 6000, dtype, seed=4)
    s.pre[17] = (s.q[0, 0] * (300 * (d_c + d_rope) ** 0.5 / s.q[0, 0].double().square().sum())).to(dtype)
    s.prefix = dict(prefix_kv=s.pre.cuda())
    s.check_all(*s.run())

"""The convolution on small integers, without SiLU: every sum and every output is exact in fp32 (and in bf16), so that a
token that is lost, doubled or taken from a neighbour shows as a whole number.  dw and dbias are sums over all tokens of
terms of at most 4 in magnitude: exact below 2^24 / 4 tokens."""
import pytest
import torch

import gated_delta_rule_91_b200 as gdr

pytestmark = pytest.mark.gpu
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def ints(g, most, *size):
    return torch.randint(-most, most + 1, size, generator=g).float()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,C,K,extra", [
    (1, 1, 8, 4, 0), (3, 2, 40, 8, 8), (2, 191, 64, 4, 0), (97, 193, 64, 4, 8), (96, 192, 64, 8, 0), (1, 100000, 8, 4, 0),
    (2, 30000, 20, 7, 4), (2, 30000, 21, 7, 0), (5000, 3, 64, 4, 0), (3, 17, 5001, 2, 0), (4, 4400, 2304, 4, 0), (1, 9000, 2304, 5, 64),
    (2, 6000, 1000, 3, 0), (300, 130, 130, 6, 0), (1, 70001, 1, 4, 0)])
def test_every_token_once(B, T, C, K, extra, dtype):
    g = torch.Generator().manual_seed(B + T + C + K)
    t = TYPES[dtype]
    x = ints(g, 2, B, T, C + extra).to(t).cuda()[..., :C]
    state, dy, ds = (ints(g, 2, B, n, C).to(t).cuda() for n in (K - 1, T, K - 1))
    w, bias = ints(g, 2, C, K).cuda(), ints(g, 3, C).cuda()
    so = torch.empty_like(state)
    y = gdr.gdr_conv_fwd(x, w, bias, conv_state=state, conv_state_out=so, silu=False)
    full = torch.cat([state, x], 1).float()
    want = bias + sum(full[:, j:j + T] * w[:, j] for j in range(K))
    assert torch.equal(y.float(), want)
    assert torch.equal(so.float(), full[:, T:])
    out = gdr.gdr_conv_bwd(x, w, dy, bias, conv_state=state, dconv_state_out=ds, silu=False)
    dfull = torch.zeros_like(full)
    for j in range(K):
        dfull[:, j:j + T] += dy.float() * w[:, j]
    dfull[:, T:] += ds.float()
    assert torch.equal(out["dx"].float(), dfull[:, K - 1:])
    assert torch.equal(out["dconv_state"].float(), dfull[:, :K - 1])
    assert torch.equal(out["dbias"], dy.double().sum((0, 1)).float())
    dw = torch.stack([(dy.double() * full[:, j:j + T].double()).sum((0, 1)) for j in range(K)], 1)
    assert torch.equal(out["dw"], dw.float())

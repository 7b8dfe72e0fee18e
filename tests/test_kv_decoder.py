"""The decode step with a mix callback (attention over the key/value cache
before each layer's FFN) against the captured step without one and against a
step-by-step evaluation with the oracles."""
import numpy as np
import pytest
import torch

import oracle
from oracle.kv import KvOracle
from tests.parity import FFN_TOL, build_decoder
from workloads import SMALL_BATCHED, SMALL_BF16, SMALL_F16, SMALL_OPT, make_workload

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from sparse_activation_decode_gb300.build import build
    build()


@pytest.mark.parametrize("cfg", [SMALL_F16, SMALL_BF16, SMALL_OPT, SMALL_BATCHED,
                                 SMALL_F16.replace(slots="compact")], ids=lambda c: f"{c.name}-{c.slots}")
def test_an_empty_mix_is_the_plain_step(cfg):
    wl = make_workload(cfg)
    a, b = build_decoder(wl), build_decoder(wl)
    seen = []
    for t in range(4):
        x, y = wl.x[t].cuda().clone(), wl.x[t].cuda().clone()
        a.decode_token(x)
        assert b.decode_token(y, mix=lambda layer, h: seen.append(layer)) is None
        torch.cuda.synchronize()
        assert a.counts() == b.counts()
        # the same FFNs, joined in another order of fp32 sums
        assert oracle.rel_l2(y.cpu().numpy().ravel(), x.cpu().numpy().ravel()) <= 1e-5
    assert seen == list(range(cfg.n_layers)) * 4
    for s in range(cfg.n_sparse):
        assert a.get_state(cfg.n_dense + s) == b.get_state(cfg.n_dense + s)
    a.close()
    b.close()


@pytest.mark.parametrize("cfg", [SMALL_BF16, SMALL_BATCHED], ids=lambda c: c.name)
def test_a_decode_step_with_attention(cfg):
    """Each layer: h += attention of h's heads over the cache, then the FFN;
    checked against the 64-bit attention and the layer-by-layer FFN calls."""
    from sparse_activation_decode_gb300 import KvCache
    B, D, dim = cfg.batch, cfg.d_model, 64
    heads, kvh = D // dim, D // dim // 2
    wl = make_workload(cfg)
    dec, ref = build_decoder(wl), build_decoder(wl)
    cache = KvCache(n_layers=cfg.n_layers, n_pages=4 * B, n_kv_heads=kvh, head_dim=dim, max_seqs=B, max_pages=4)
    orc = KvOracle(cfg.n_layers, 4 * B, kvh, dim, B, 4)
    one = torch.ones(B, dtype=torch.int32, device="cuda")

    def mix(layer, h):
        assert torch.cuda.current_stream() == dec.main_stream
        x = h.view(B, heads, dim)
        if layer == 0:
            cache.reserve(one)
        cache.append(layer, x[:, :kvh], x[:, kvh:])
        h += 0.1 * cache.attend(layer, x, window=3, sinks=1).reshape(h.shape)

    for t in range(5):
        h = wl.x[t].cuda().clone()
        dec.decode_token(h, mix=mix)
        # the same step with the oracle's attention in 64 bits
        g = wl.x[t].cuda().clone().reshape(B, D)
        orc.reserve([1] * B)
        ids = None
        for layer in range(cfg.n_layers):
            x = g.double().cpu().numpy().reshape(B, heads, dim)
            orc.append(layer, x[:, :kvh].astype(np.float32).astype(np.float64), x[:, kvh:], [1] * B)
            y, _, _ = orc.attend(layer, x, [1] * B, 1 / np.sqrt(dim), window=3, sinks=1)
            g = (g.double().cpu() + 0.1 * torch.from_numpy(y).reshape(B, D)).float().cuda()
            if layer >= cfg.n_dense:
                ref.scatter(layer)
            g = ref.ffn_layers(layer, 1, g)
            if layer == 0:
                ids = ref.predict(g)
                ref.delta(ids, -1)
        torch.cuda.synchronize()
        assert oracle.rel_l2(h.cpu().numpy().ravel(), g.cpu().numpy().ravel()) <= FFN_TOL
    cache.check()
    dec.check_error()
    dec.close()
    ref.close()


def test_mix_refusals():
    cfg = SMALL_F16
    wl = make_workload(cfg)
    dec = build_decoder(wl)
    h = wl.x[0].cuda().clone()
    for kw, x in ((dict(stats=True), h), ({}, h[:, :64]), ({}, h.double()), ({}, h.cpu())):
        with pytest.raises(ValueError):
            dec.decode_token(x, mix=lambda layer, y: None, **kw)
    dec.close()
    opt = make_workload(SMALL_OPT.replace(lookahead=1))
    dec = build_decoder(opt)
    with pytest.raises(ValueError):
        dec.decode_token(opt.x[0].cuda().clone(), mix=lambda layer, y: None)
    dec.close()


@pytest.mark.parametrize("cfg", [SMALL_F16, SMALL_OPT, SMALL_F16.replace(slots="compact")],
                         ids=lambda c: f"{c.name}-{c.slots}")
def test_a_mix_that_raises_leaves_a_decoder_that_goes_on(cfg):
    wl = make_workload(cfg)
    a, b = build_decoder(wl), build_decoder(wl)
    for t in range(3):
        for stop in (0, 1, cfg.n_layers - 1):
            def mix(layer, h):
                if layer == stop:
                    raise KeyError(layer)
            with pytest.raises(KeyError):
                b.decode_token(wl.x[t].cuda().clone(), mix=mix)
        x, y = wl.x[t].cuda().clone(), wl.x[t].cuda().clone()
        a.decode_token(x)
        b.decode_token(y, mix=(lambda layer, h: None) if t == 1 else None)
        torch.cuda.synchronize()
        assert oracle.rel_l2(y.cpu().numpy().ravel(), x.cpu().numpy().ravel()) <= 1e-5
    a.close()
    b.close()

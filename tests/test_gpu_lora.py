"""LinearLora on the GPU against the FP64 oracle, within the layer's bound (8e-3 |y| + 1e-3
rms(y): the second product's own error, at most 2^-17 of its terms, is far inside it)."""
import numpy as np
import pytest

from oracle import decoder_ops as do
from weight_only_bit_q4_gb300 import q4lin, synth

from gpu_util import assert_close, to_dev, torch, x_to_dev, y_bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from weight_only_bit_q4_gb300 import build
    build.build()
    q4lin.load()
    assert q4lin.clear_device_status() == 0
    yield
    assert q4lin.device_status() == 0


def bits(shape, seed, std):
    n = int(np.prod(shape))
    return synth.to_bf16_bits(synth.normal(synth.stream_state(seed, 0x4C6F), n) * std).reshape(shape)


def problem(N, K, T, L, R, seed, ids=None):
    wq, s, x = synth.make_problem(N, K, T, w_seed=seed, x_seed=seed + 1)
    a, b = bits((L, R, K), seed + 2, K ** -0.5), bits((L, N, R), seed + 3, 0.5)
    rng = np.random.default_rng(seed)
    if ids is None:
        ids = rng.integers(-1, L, size=T)
    sc = rng.uniform(0.5, 2.0, size=L).astype(np.float32)
    return wq, s, x, a, b, np.asarray(ids, dtype=np.int32), sc


def call(p, ranks=None, **kw):
    t = torch()
    wq, s, x, a, b, ids, sc = p
    d = to_dev(wq, s, x)
    rk = None if ranks is None else t.from_numpy(np.asarray(ranks, dtype=np.int32)).cuda()
    y = q4lin.linear_lora(*d, x_to_dev(a), x_to_dev(b), t.from_numpy(ids).cuda(),
                          None if sc is None else t.from_numpy(sc).cuda(), rk, **kw)
    t.cuda.synchronize()
    return y


SHAPES = [(6144, 5120, 1, 4, 16), (77, 72, 1, 1, 8), (1000, 1160, 1, 3, 64), (33, 17408, 1, 2, 256), (300, 640, 2, 5, 16),
          (300, 640, 7, 5, 24), (129, 4104, 8, 9, 16), (6144, 5120, 9, 3, 32), (500, 1992, 17, 20, 64), (40, 136, 25, 3, 256),
          (2000, 2048, 32, 40, 16), (300, 640, 33, 5, 16), (1000, 1160, 75, 16, 64), (129, 264, 257, 3, 8),
          (640, 2048, 600, 4, 72), (1, 8, 1, 1, 8), (1, 8, 40, 2, 8)]


@pytest.mark.parametrize("N,K,T,L,R", SHAPES)
def test_matches_oracle(N, K, T, L, R):
    p = problem(N, K, T, L, R, N + T)
    y = call(p)
    assert_close(y_bits(y), do.linear_lora(*p), f"lora {N}x{K} T={T} L={L} R={R}")
    assert np.array_equal(y_bits(call(p)), y_bits(y))   # deterministic


@pytest.mark.parametrize("T", [1, 6, 20, 50])
def test_ranks_and_unused_garbage(T):
    """Ranks 0, odd, negative and too large; what lies past a rank is NaN and must not show."""
    N, K, L, R = 200, 520, 6, 24
    ranks = [0, 5, 24, -3, 99, 17]
    p = problem(N, K, T, L, R, 5 + T, ids=np.arange(T) % (L + 1) - (T == 20))
    a, b = p[3].copy(), p[4].copy()
    for i, r in enumerate(ranks):
        r = min(max(r, 0), R)
        a[i, r:], b[i, :, r:] = 0x7FC0, 0x7FC0
    q = p[:3] + (a, b) + p[5:]
    assert_close(y_bits(call(q, ranks)), do.linear_lora(*p, ranks), f"ranks T={T}")


@pytest.mark.parametrize("T", [1, 8, 40])
def test_without_any_adapter_is_the_projection(T):
    p = problem(300, 640, T, 2, 16, 9, ids=np.where(np.arange(T) % 2, -1, 1 << 30))
    y = call(p)
    t = torch()
    base = q4lin.linear(*to_dev(*p[:3]))
    t.cuda.synchronize()
    if T != 40:
        assert np.array_equal(y_bits(y), y_bits(base))
    assert_close(y_bits(y), do.linear_lora(*p), "no adapter")
    for L, R in ((0, 16), (2, 0)):   # no adapters at all
        q = p[:3] + (p[3][:L, :R], p[4][:L, :, :R]) + p[5:6] + (p[6][:L],)
        assert np.array_equal(y_bits(call(q)), y_bits(base))


@pytest.mark.parametrize("T", [1, 5, 24, 64])
def test_output_window_stream_and_graph(T):
    t = torch()
    N, K, L, R = 200, 1024, 3, 16
    p = problem(N, K, T, L, R, 21)
    d = to_dev(*p[:3])
    a, b, ids, sc = x_to_dev(p[3]), x_to_dev(p[4]), t.from_numpy(p[5]).cuda(), t.from_numpy(p[6]).cuda()
    buf = t.full((512 + T * N + 512,), -3.0, dtype=t.bfloat16, device="cuda")
    y = buf[512:512 + T * N].view(T, N)
    ws = t.empty(q4lin.lora_workspace_bytes(N, K, T, L, R), dtype=t.uint8, device="cuda")
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    q4lin.linear_lora(*d, a, b, ids, sc, y=y, workspace=ws, stream=stream)
    stream.synchronize()
    want = do.linear_lora(*p)
    assert_close(y_bits(y), want, "window")
    assert bool((buf[:512] == -3.0).all()) and bool((buf[512 + T * N:] == -3.0).all())
    y.zero_()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        q4lin.linear_lora(*d, a, b, ids, sc, y=y, workspace=ws)
    ids.copy_(t.from_numpy((p[5] + 1) % L).int())   # the graph reads the ids of the moment
    g.replay()
    t.cuda.synchronize()
    assert_close(y_bits(y), do.linear_lora(*p[:5], (p[5] + 1) % L, p[6]), "replay")


def test_chained_calls_share_one_workspace():
    """Calls that follow one another in a stream, each reading what the one before wrote."""
    t = torch()
    N = K = 512
    L, R = 2, 16
    ws = t.empty(1 << 24, dtype=t.uint8, device="cuda")
    for T in (1, 4, 12, 40):
        p = problem(N, K, T, L, R, 31 + T)
        d = to_dev(*p[:3])
        args = (x_to_dev(p[3]), x_to_dev(p[4]), t.from_numpy(p[5]).cuda(), t.from_numpy(p[6]).cuda())
        y1, y2 = t.empty_like(d[2]), t.empty_like(d[2])
        for _ in range(20):
            q4lin.linear_lora(*d, *args, y=y1, workspace=ws)
            y1.mul_(1.0 / 64)
            q4lin.linear_lora(d[0], d[1], y1, *args, y=y2, workspace=ws)
        t.cuda.synchronize()
        x2 = y1.view(t.int16).cpu().numpy().view(np.uint16)
        assert_close(y_bits(y2), do.linear_lora(p[0], p[1], x2, *p[3:]), f"chained T={T}")


def test_wrapper_refuses():
    t = torch()
    p = problem(64, 128, 2, 2, 8, 3)
    d = to_dev(*p[:3])
    a, b, ids = x_to_dev(p[3]), x_to_dev(p[4]), t.from_numpy(p[5]).cuda()
    with pytest.raises(ValueError):
        q4lin.linear_lora(*d, a, b, ids.long())
    with pytest.raises(ValueError):
        q4lin.linear_lora(*d, a, b.transpose(1, 2), ids)
    with pytest.raises(ValueError):
        q4lin.linear_lora(*d, a, b, ids, workspace=t.empty(16, dtype=t.uint8, device="cuda"))
    with pytest.raises(q4lin.Q4LinError):
        q4lin.linear_lora(*d, a[:, :4].contiguous(), b[:, :, :4].contiguous(), ids)

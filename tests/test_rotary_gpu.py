"""Rotary positions, their gradient and the cache insertion against a 64-bit implementation.

Tolerance of a bf16 result: half a step, 2^-8 of the value, and the fp32 rotation before it: cosine and sine
are off by less than 2^-21 (the angle's reduction 2^-24 of a turn, the function's own error), two products
and a sum by 3 * 2^-24 of the pair's magnitude; 2^-20 (|a| + |b|) covers both."""
import pytest
import torch

import _serving as S
import block_sparse_attention_08_gb300 as msa

pytestmark = pytest.mark.gpu

FORMS = [(128, 1, False), (128, 3, False), (128, 3, True), (64, 3, False), (64, 1, True), (16, 2, False), (16, 1, True),
         (48, 4, True), (80, 3, False), (112, 1, False)]


def _setup(tokens, rot, num_axes, seed=0, far=1000):
    gen = torch.Generator("cuda").manual_seed(seed)
    positions = torch.randint(far, (num_axes, tokens), generator=gen, device="cuda", dtype=torch.int32)
    inv_freq = torch.tensor([1e6 ** (-2.0 * j / rot) for j in range(rot // 2)], device="cuda")
    axes = tuple(int(a) for a in torch.randint(num_axes, (rot // 2,), generator=torch.Generator().manual_seed(seed)))
    return gen, positions, inv_freq, axes


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").bfloat16()


def _close(got, ref, x, rot, interleaved):
    """ref: the float64 rotation of x."""
    m = x.detach().double().abs()
    pair = torch.zeros_like(m)
    half = rot // 2
    if interleaved:
        pair[..., :rot] = m[..., :rot].unflatten(-1, (half, 2)).sum(-1, keepdim=True).expand(*m.shape[:-1], half, 2).flatten(-2)
    else:
        pair[..., :rot] = (m[..., :half] + m[..., half:rot]).repeat(1, 1, 2)
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * pair
    assert bool(((got.double() - ref).abs() <= tol).all())
    assert torch.equal(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("rot,num_axes,interleaved", FORMS)
def test_rotary_and_its_gradient(rot, num_axes, interleaved):
    for tokens, qh, kh in ((1, 64, 4), (3, 4, 1), (130, 64, 4), (257, 7, 33)):
        gen, positions, inv_freq, axes = _setup(tokens, rot, num_axes, seed=tokens)
        q, k = _randn(gen, tokens, qh, 128).requires_grad_(), _randn(gen, tokens, kh, 128).requires_grad_()
        qo, ko = msa.rotary(q, k, positions, inv_freq, axes=axes, interleaved=interleaved)
        for x, y in ((q, qo), (k, ko)):
            _close(y, S.rotate(x, positions, inv_freq, axes, interleaved), x, rot, interleaved)
        gq, gk = _randn(gen, *q.shape), _randn(gen, *k.shape)
        dq, dk = torch.autograd.grad((qo, ko), (q, k), (gq, gk))
        for x, y in ((gq, dq), (gk, dk)):
            _close(y, S.rotate(x, positions, inv_freq, axes, interleaved, -1), x, rot, interleaved)


def test_gradient_against_differences():
    # the map is linear, so a difference over a large step is its derivative but for the roundings: of both outputs and
    # of the gradient, 2^-8 each, summed over the pair's two members
    gen, positions, inv_freq, axes = _setup(5, 64, 3)
    q, g = _randn(gen, 5, 4, 128), _randn(gen, 5, 4, 128)
    leaf = q.clone().requires_grad_()
    out, _ = msa.rotary(leaf, q[:, :1].contiguous(), positions, inv_freq, axes=axes)
    (dq,) = torch.autograd.grad(out, leaf, g)
    for t, h, d in ((0, 0, 0), (4, 3, 31), (2, 1, 32), (3, 2, 63), (1, 0, 64), (4, 0, 127)):
        up, down = q.clone(), q.clone()
        up[t, h, d], down[t, h, d] = 4.0, -4.0
        diff = (msa.msa_rotary(up, None, positions, inv_freq, axes=axes)[0].double()
                - msa.msa_rotary(down, None, positions, inv_freq, axes=axes)[0].double()) / 8.0
        num = float((diff * g.double()).sum())
        tol = 2.0 ** -8 * (abs(num) + 3 * float(g.double().abs().max()) * (4 + float(q.double().abs().max())))
        assert abs(num - float(dq[t, h, d])) <= tol


def test_many_tokens_through_the_ring():
    # more tokens than CTAs and stages: every CTA's ring goes round several times
    gen, positions, inv_freq, axes = _setup(6007, 64, 3)
    q, k = _randn(gen, 6007, 64, 128), _randn(gen, 6007, 4, 128)
    qo, ko = msa.msa_rotary(q, k, positions, inv_freq, axes=axes)
    _close(qo, S.rotate(q, positions, inv_freq, axes, False), q, 64, False)
    _close(ko, S.rotate(k, positions, inv_freq, axes, False), k, 64, False)
    qkv = torch.cat([q, k, k.flip(0)], 1)
    slots = torch.randperm(6144, generator=gen, device="cuda")[:6007]
    k_cache, v_cache = (torch.zeros(6144, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = msa.msa_rotary_insert(qkv[:, :64], qkv[:, 64:68], qkv[:, 68:], positions, inv_freq, slots, k_cache, v_cache,
                                axes=axes)
    assert torch.equal(got, qo) and torch.equal(k_cache[slots], ko) and torch.equal(v_cache[slots], k.flip(0))


def test_differentiated_twice():
    gen, positions, inv_freq, axes = _setup(9, 128, 2)
    q, k = _randn(gen, 9, 64, 128).requires_grad_(), _randn(gen, 9, 4, 128).requires_grad_()
    g = _randn(gen, 9, 64, 128).requires_grad_()
    out, _ = msa.rotary(q, k, positions, inv_freq, axes=axes)
    (dq,) = torch.autograd.grad(out, q, g, create_graph=True)
    h = _randn(gen, 9, 64, 128)
    (dg,) = torch.autograd.grad(dq, g, h)
    assert torch.equal(dg, msa.msa_rotary(h, None, positions, inv_freq, axes=axes)[0])
    with pytest.raises(TypeError):
        msa.rotary(q, None, positions, inv_freq)


@pytest.mark.parametrize("far", [2 ** 20, 2 ** 24 + 1000, 2 ** 31 - 1])
def test_far_positions_keep_their_angle(far):
    gen, positions, inv_freq, axes = _setup(64, 128, 2, far=far)
    positions[0, 0], positions[1, 1], positions[0, 2] = far - 1, -far + 1, 0
    q = _randn(gen, 64, 64, 128)
    y, none = msa.msa_rotary(q, None, positions, inv_freq, axes=axes)
    assert none is None
    _close(y, S.rotate(q, positions, inv_freq, axes, False), q, 128, False)


def test_in_place_and_one_axis_vector():
    gen, positions, inv_freq, _ = _setup(33, 128, 1)
    q, k = _randn(gen, 33, 64, 128), _randn(gen, 33, 4, 128)
    want = msa.msa_rotary(q, k, positions, inv_freq)
    a, b = q.clone(), k.clone()
    msa.msa_rotary(a, b, positions[0], inv_freq, q_out=a, k_out=b)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens,rot,num_axes,interleaved", [(1, 128, 1, False), (5, 64, 3, False), (131, 128, 3, True),
                                                             (1000, 96, 2, False)])
def test_insertion(tokens, rot, num_axes, interleaved, fp8):
    gen, positions, inv_freq, axes = _setup(tokens, rot, num_axes, seed=3)
    qkv = _randn(gen, tokens, 72, 128)
    q, k, v = qkv[:, :64], qkv[:, 64:68], qkv[:, 68:]
    num = 128 * (tokens // 128 + 3)
    slots = torch.randperm(num, generator=gen, device="cuda")[:tokens]
    if tokens > 4:
        slots[2], slots[4] = -1, -7  # rows that are not inserted
    ks, vs = (0.37, 0.004) if fp8 else (1.0, 1.0)  # 0.004: values past 448 scales
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    k_cache, v_cache = _randn(gen, num, 4, 128).to(dt), _randn(gen, num, 4, 128).to(dt)
    k0, v0 = k_cache.clone(), v_cache.clone()
    ko = torch.empty(tokens, 4, 128, dtype=torch.bfloat16, device="cuda")
    ws = msa.Workspace(256)
    qo = msa.msa_rotary_insert(q, k, v, positions, inv_freq, slots, k_cache, v_cache, axes=axes,
                               interleaved=interleaved, k_scale=ks, v_scale=vs, k_out=ko, workspace=ws)
    assert ws.read_device_error()[0] == 0
    _close(qo, S.rotate(q, positions, inv_freq, axes, interleaved), q, rot, interleaved)
    want_k = S.rotate(k, positions, inv_freq, axes, interleaved)
    _close(ko, want_k, k, rot, interleaved)
    live = slots >= 0
    untouched = torch.ones(num, dtype=torch.bool, device="cuda")
    untouched[slots[live]] = False
    bits = torch.uint8 if fp8 else torch.int16
    assert torch.equal(k_cache.view(bits)[untouched], k0.view(bits)[untouched])
    assert torch.equal(v_cache.view(bits)[untouched], v0.view(bits)[untouched])
    got_k, got_v = k_cache[slots[live]].double(), v_cache[slots[live]].double()
    if not fp8:
        assert torch.equal(got_v, v[live].double())
        _close(k_cache[slots[live]], want_k[live], k[live], rot, interleaved)
        return
    # E4M3: half a step is 2^-4 of a normal value, 2^-10 below 2^-6; 1e-5 for the fp32 rotation and quotient (the pair's
    # magnitude is at most 12 here)
    for got, want, scale in ((got_k, want_k[live], ks), (got_v, v[live].double(), vs)):
        want = (want / scale).clamp(-448, 448)
        assert bool(((got - want).abs() <= 2.0 ** -4 * want.abs() + 2.0 ** -10 + 1e-5 / scale).all())
    exact = (v[live].float() / torch.tensor(vs, device="cuda")).clamp(-448, 448).to(dt)
    assert torch.equal(v_cache[slots[live]].view(bits), exact.view(bits))


def test_bad_slots_and_nonfinite_values():
    gen, positions, inv_freq, axes = _setup(6, 128, 1)
    q, k, v = _randn(gen, 6, 64, 128), _randn(gen, 6, 4, 128), _randn(gen, 6, 4, 128)
    v[1, 0, 0], v[1, 0, 1], v[1, 0, 2] = float("nan"), float("inf"), float("-inf")
    k_cache, v_cache = (torch.zeros(128, 4, 128, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    slots = torch.tensor([0, 1, 128, 3, 2 ** 40, -1], device="cuda")
    ws = msa.Workspace(256)
    msa.msa_rotary_insert(q, k, v, positions, inv_freq, slots, k_cache, v_cache, axes=axes, workspace=ws)
    code, row = ws.read_device_error()
    assert code == 1 and row in (2, 4)
    rows = v_cache.float().abs().sum((1, 2)).nan_to_num(1.0) > 0
    assert rows.nonzero().flatten().tolist() == [0, 1, 3]
    x = v_cache[1, 0, :3].float()
    assert torch.isnan(x[0]) and x[1] == 448 and x[2] == -448


def test_captured_and_on_another_stream():
    gen, positions, inv_freq, axes = _setup(300, 128, 3)
    q, k, v = _randn(gen, 300, 64, 128), _randn(gen, 300, 4, 128), _randn(gen, 300, 4, 128)
    caches = [torch.zeros(512, 4, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    slots = torch.randperm(512, generator=gen, device="cuda")[:300]
    want = msa.msa_rotary_insert(q, k, v, positions, inv_freq, slots, caches[0], caches[1], axes=axes)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = msa.msa_rotary_insert(q, k, v, positions, inv_freq, slots, caches[2], caches[3], axes=axes)
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])


def test_captured_backward():
    gen, positions, inv_freq, axes = _setup(200, 128, 3)
    q, k = _randn(gen, 200, 64, 128).requires_grad_(), _randn(gen, 200, 4, 128).requires_grad_()
    g = _randn(gen, 200, 64, 128), _randn(gen, 200, 4, 128)

    def step():
        return torch.autograd.grad(msa.rotary(q, k, positions, inv_freq, axes=axes), (q, k), g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [x.clone() for x in step()]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gradient_of_one_output_and_refusals():
    gen = torch.Generator("cuda").manual_seed(9)
    q = torch.randn(5, 64, 128, generator=gen, device="cuda").bfloat16().requires_grad_()
    k = torch.randn(5, 4, 128, generator=gen, device="cuda").bfloat16().requires_grad_()
    pos = torch.arange(5, device="cuda", dtype=torch.int32)
    inv = torch.ones(16, device="cuda")
    qo, ko = msa.rotary(q, k, pos, inv)
    g = torch.randn(5, 64, 128, generator=gen, device="cuda").bfloat16()
    gq, gk = torch.autograd.grad(qo, (q, k), g, allow_unused=True)
    assert torch.equal(gq, msa.msa_rotary(g, None, pos, inv, inverse=True)[0])
    assert gk is None or not gk.any()
    # a gradient that is one value for all, and one of another layout
    gq, gk = torch.autograd.grad(msa.rotary(q, k, pos, inv), (q, k),
                                 (torch.ones(1, 1, 1, device="cuda").bfloat16().expand(5, 64, 128),
                                  torch.ones(128, 4, 5, device="cuda").bfloat16().permute(2, 1, 0)))
    one = msa.msa_rotary(torch.ones_like(q), torch.ones_like(k), pos, inv, inverse=True)
    assert torch.equal(gq, one[0]) and torch.equal(gk, one[1])
    odd = torch.randn(5 * 64 * 128 + 3, generator=gen, device="cuda").bfloat16()[3:].view(5, 64, 128)  # 6 bytes off
    (gq,) = torch.autograd.grad(msa.rotary(q, k, pos, inv)[0], q, odd)
    assert torch.equal(gq, msa.msa_rotary(odd.clone(), None, pos, inv, inverse=True)[0])
    with torch.no_grad():
        assert not msa.rotary(q, k, pos, inv)[0].requires_grad
    with pytest.raises(msa.MsaError):
        msa.rotary(q, k, pos, torch.ones(12, device="cuda"))  # 24 dims: not a multiple of 16
    with pytest.raises(msa.MsaError):
        msa.rotary(q, k, pos.repeat(5, 1), inv)  # five axes
    with pytest.raises(ValueError):
        msa.rotary(q, k.cpu(), pos, inv)
    with pytest.raises(TypeError):
        msa.rotary(q, None, pos, inv)
    # refused calls leave no error behind
    assert torch.equal(msa.rotary(q, k, pos, inv)[0], qo)

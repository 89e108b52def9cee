"""grad_clip of more tensors than a launch names and more bytes than the last-level
cache holds, as a whole model's gradients are: every element against float64.

The coefficient takes two roundings (max_norm to float32 and its own), the product
one: 3.1 u of an element, u = 2^-24, and half a step of bfloat16."""
import math

import pytest
import torch

from tests.gpu_util import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def tensors(count, total, dtypes, seed):
    """Views one after the other from element 3 (5) of a buffer a type, with a gap
    of one element behind every tenth; the buffers too."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    share = [1 + (7919 * i) % 97 for i in range(count)]
    sizes = [total * s // sum(share) + i % 5 for i, s in enumerate(share)]
    buf = {t: torch.empty(sum(sizes) + count + 64, device="cuda").normal_(0, 1e-2, generator=g).to(t)
           for t in dtypes}
    at, out = {t: 3 if t == F32 else 5 for t in dtypes}, []
    for i, n in enumerate(sizes):
        t = dtypes[i % len(dtypes)]
        out.append(buf[t][at[t]:at[t] + n])
        at[t] += n + (i % 10 == 9)
    return out, buf


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("dtypes", [(F32,), (BF16,), (F32, BF16)])
@pytest.mark.parametrize("count, total", [(300, 140_000_000), (113, 70_000_000), (112, 150_000_000),
                                          (448, 1_000_000)])
def test_many(gpu_lib, count, total, dtypes, apart):
    announce(f"grad_clip {count} tensors, {total} elements, {dtypes}, apart={apart}")
    grads, buf = tensors(count, total, dtypes, count)
    before = {t: b.clone() for t, b in buf.items()}
    was = [g.clone() for g in grads]
    ref = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    norm = torch.empty(1, device="cuda")
    out, to = (tensors(count, total, dtypes, 99) if apart else (grads, buf))
    kept = {t: b.clone() for t, b in to.items()}
    gpu_lib.grad_clip(grads, 0.3 * ref, norm, out=out if apart else None)
    assert abs(float(norm) - ref) <= 1.001 * U * ref
    coef = 0.3 * ref / (ref + 1e-6)
    for o, w in zip(out, was):
        want = w.double() * coef
        tol = want.abs() * (3.1 * U + (2.0 ** -8 if w.dtype == BF16 else 0.0)) + 1e-37
        assert bool(((o.double() - want).abs() <= tol).all())
    for t, b in to.items():                                # nothing between the views changed
        k, cover = kept[t], torch.ones_like(b, dtype=torch.bool)
        for o in out:
            if o.dtype == t:
                a = (o.data_ptr() - b.data_ptr()) // b.element_size()
                cover[a:a + o.numel()] = False
        assert torch.equal(b[cover], k[cover])
    if apart:
        assert all(torch.equal(b, before[t]) for t, b in buf.items())
    del grads, out, buf, to, before, kept, was
    torch.cuda.empty_cache()

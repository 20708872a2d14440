"""Refusals of the latent attention's entry points, on the host and before
anything is enqueued: no GPU is needed."""
import ctypes

import pytest
import torch

import gated_delta_rule_21_gb300 as kda
from gated_delta_rule_21_gb300 import build as kbuild

FAKE = 0x10000      # 256-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    kbuild.build()
    return kda.lib()


def rotate(L, B=1, T=4, H=2, dim=64, dtype=1, x=FAKE, pos=None, freq=FAKE, y=FAKE):
    d = kda.kda_rotate_desc(B, T, H, dim, dtype, 1, 0, 512, 128, 64, 512, 128, 64)
    return L.kda_rotate(d, x, pos, freq, y, None)


@pytest.mark.parametrize("kw,want", [
    (dict(x=None), 1), (dict(freq=None), 1), (dict(y=None), 1), (dict(B=0), 1), (dict(T=0), 1),
    (dict(H=0), 1), (dict(dim=0), 1), (dict(dtype=2), 1), (dict(dim=7), 2), (dict(dim=258), 2),
    (dict(B=1 << 16, T=1 << 16), 2), (dict(H=1 << 20), 2), (dict(x=FAKE + 1), 3),
    (dict(dtype=0, y=FAKE + 2), 3), (dict(freq=FAKE + 2), 3), (dict(pos=FAKE + 1), 3)])
def test_rotate_refuses(L, kw, want):
    assert rotate(L, **kw) == want


def cache_shape(B=2, T=1, H=4, pages=8, n_pages=20, page=64, C=512, R=64, dtype=1):
    return kda.kda_latent_cache(B, T, H, pages, n_pages, page, C, R, dtype, page * (C + R), C + R,
                                T * H * C, H * C, C, T * H * R, H * R, R, T * C, C, T * R, R)


def append(L, latent=FAKE, k=FAKE, q=None, freq=FAKE, table=FAKE, lengths=FAKE, new=None,
           cache=FAKE, out=None, **shape):
    return L.kda_latent_append(cache_shape(**shape), latent, k, q, freq, 1, table, lengths, new,
                               cache, out, None)


@pytest.mark.parametrize("kw,want", [
    (dict(latent=None), 1), (dict(k=None), 1), (dict(table=None), 1), (dict(lengths=None), 1),
    (dict(cache=None), 1), (dict(q=FAKE), 1), (dict(out=FAKE), 1),
    (dict(q=FAKE, out=FAKE, freq=None), 1), (dict(R=0), 1), (dict(R=0, k=None), 1),
    (dict(B=0), 1), (dict(T=0), 1), (dict(pages=0), 1), (dict(n_pages=0), 1), (dict(page=0), 1),
    (dict(C=0), 1), (dict(R=-2), 1), (dict(dtype=4), 1), (dict(C=5000), 2), (dict(R=63), 2),
    (dict(R=300), 2), (dict(latent=FAKE + 1), 3), (dict(dtype=0, cache=FAKE + 2), 3),
    (dict(table=FAKE + 2), 3)])
def test_append_refuses(L, kw, want):
    assert append(L, **kw) == want


def step(L, q=FAKE, r=FAKE, cache=FAKE, table=FAKE, lengths=FAKE, scale=0.1, o=FAKE, lse=None,
         ws=FAKE, nbytes=1 << 30, impl=0, **shape):
    return L.kda_latent_step(cache_shape(**shape), q, r, cache, table, lengths, None, scale, o,
                             lse, ws, nbytes, impl, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), 1), (dict(r=None), 1), (dict(R=0), 1), (dict(cache=None), 1),
    (dict(table=None), 1), (dict(lengths=None), 1), (dict(o=None), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(impl=3), 1),
    (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(page=0), 1), (dict(dtype=9), 1),
    (dict(C=384), 2), (dict(C=96), 2), (dict(R=16), 2), (dict(R=128), 2),
    (dict(T=1 << 12, H=1 << 12), 2), (dict(pages=1 << 20, page=1 << 12), 2),
    (dict(impl=2, dtype=0), 2), (dict(impl=2, page=48), 2), (dict(impl=2, page=4), 2),
    (dict(impl=2, cache=FAKE + 2), 2),
    (dict(q=FAKE + 1), 3), (dict(o=FAKE + 8), 3), (dict(lse=FAKE + 2), 3), (dict(ws=FAKE + 64), 3),
    (dict(ws=None), 4), (dict(nbytes=1000), 4)])
def test_step_refuses(L, kw, want):
    assert step(L, **kw) == want


def latent_shape(B=1, T=64, H=4, K=128, R=64, V=128, dtype=1, qt=None):
    return kda.kda_latent_shape(B, T, H, K, R, V, dtype, T * H * K, qt or H * K, K, T * H * R,
                                H * R, R, T * H * K, H * K, K, T * R, R, T * H * V, H * V, V)


def fwd(L, q=FAKE, r=FAKE, k=FAKE, kr=FAKE, v=FAKE, scale=0.1, seg=None, o=FAKE, lse=None,
        ws=FAKE, nbytes=1 << 30, impl=0, **shape):
    return L.kda_latent_fwd(latent_shape(**shape), q, r, k, kr, v, scale, seg, o, lse, ws, nbytes,
                            impl, None)


COMMON = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(r=None), 1),
    (dict(kr=None), 1), (dict(R=0), 1), (dict(scale=float("nan")), 1), (dict(impl=3), 1),
    (dict(B=0), 1), (dict(T=0), 1), (dict(H=0), 1), (dict(dtype=2), 1), (dict(K=96), 2),
    (dict(V=256), 2), (dict(R=16), 2), (dict(B=1 << 10, T=1 << 14, H=1), 2),
    (dict(impl=2, dtype=0), 2), (dict(impl=2, scale=-0.1), 2), (dict(q=FAKE + 1), 3),
    (dict(o=FAKE + 8), 3), (dict(lse=FAKE + 2), 3), (dict(impl=2, q=FAKE + 2), 3), (dict(impl=2, qt=515), 3),
    (dict(seg=FAKE + 2), 3), (dict(ws=FAKE + 64), 3), (dict(ws=None), 4), (dict(nbytes=255), 4)]


@pytest.mark.parametrize("kw,want", COMMON + [(dict(o=None), 1)])
def test_fwd_refuses(L, kw, want):
    assert fwd(L, **kw) == want


def bwd(L, q=FAKE, r=FAKE, k=FAKE, kr=FAKE, v=FAKE, scale=0.1, seg=None, o=FAKE, lse=FAKE,
        d_o=FAKE, dq=FAKE, dqr=FAKE, dk=FAKE, dkr=FAKE, dv=FAKE, ws=FAKE, nbytes=1 << 30, impl=0,
        **shape):
    return L.kda_latent_bwd(latent_shape(**shape), q, r, k, kr, v, scale, seg, o, lse, d_o, dq,
                            dqr, dk, dkr, dv, ws, nbytes, impl, None)


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(o=None), 1), (dict(lse=None), 1), (dict(d_o=None), 1), (dict(dq=None), 1),
    (dict(dqr=None), 1), (dict(dkr=None), 1), (dict(R=0, r=None, kr=None), 1),
    (dict(dk=FAKE + 8), 3), (dict(nbytes=40000), 4)])
def test_bwd_refuses(L, kw, want):
    assert bwd(L, **kw) == want


def test_workspace_sizes(L):
    # header, two tables of 4 bytes a token; backward also 4 bytes a token and head
    # and each head's part of dk_rope
    assert kda.latent_workspace_size(1, 64, 4, 64) == 256 + 2 * 256
    assert kda.latent_workspace_size(1, 64, 4, 64, backward=True) == \
        256 + 2 * 256 + 1024 + 64 * 4 * 64 * 4
    assert kda.latent_workspace_size(1, 64, 4, 48) == 0
    assert kda.latent_step_workspace_size(1, 1, 4, 500) == 0
    assert kda.latent_step_workspace_size(3, 1, 4, 512) == \
        kda.latent_step_workspace_size(1, 5, 64, 512)      # of one part for each SM
    assert ctypes.sizeof(kda.kda_latent_cache) == 136
    assert ctypes.sizeof(kda.kda_latent_shape) == 144
    assert ctypes.sizeof(kda.kda_rotate_desc) == 80


def test_a_call_goes_to_its_tensors_device(monkeypatch):
    """Whichever device is current; with a stream, to the stream."""
    import contextlib

    class Far:
        is_cuda = True

        def get_device(self):
            return 1

    seen = []

    @contextlib.contextmanager
    def entered(where):
        seen.append(where)
        yield

    monkeypatch.setattr(kda, "_device_now", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", entered)
    monkeypatch.setattr(torch.cuda, "stream", entered)
    assert kda._away(Far(), None) and not kda._away(torch.zeros(2), None)
    assert kda._moved(lambda a, b: (a, b), Far(), None, 5, b=6) == (5, 6) and seen == [1]
    assert kda._moved(lambda a: a, Far(), "its stream", 7) == 7 and seen == [1, "its stream"]
    monkeypatch.setattr(kda, "_device_now", lambda: 1)
    assert not kda._away(Far(), None)


def test_python_checks_come_before_the_library():
    x = torch.zeros(1, 4, 2, 32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.rotate(x, torch.zeros(16))
    with pytest.raises(ValueError, match="CUDA"):
        kda.latent_append(x[:, :, 0], None, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.latent_step(x, None, x, x, x, scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        kda.latent_fwd(x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        kda.latent_bwd(x, x, x, x, x, x)
    with pytest.raises(TypeError, match="scale"):
        kda.latent_step(x, None, x, x, x)

"""A decoding step's operators have no derivatives, and say so wherever one would get lost: kv_rotate,
kv_append_rotated, sample_rows."""
import warnings

import pytest
import torch

import _kv

pytestmark = pytest.mark.gpu
F16 = torch.float16


@pytest.fixture(scope="module")
def tk():
    import topk_selection_gb300

    yield topk_selection_gb300
    topk_selection_gb300.check_stream()


def rotation():
    freq = (1000.0 ** (-torch.arange(32) / 32)).cuda()
    return dict(x=torch.randn(3, 2, 64, device="cuda").to(F16), pos=torch.arange(3, dtype=torch.int32, device="cuda"),
                freq=freq, norm=torch.ones(64, dtype=F16, device="cuda"))


def appending(tk, a, **kw):
    cache = _kv.Cache([9, 3, 0], 2, 64, 16, F16, "head", room=4, seed=1)
    k, v, table, lens = cache.dev()
    args = dict(k_new=a["x"], v_new=a["x"].detach().clone(), freq=a["freq"], q=a["x"].detach().clone(), k_norm=a["norm"],
                q_norm=a["norm"])
    args.update(kw)
    return tk.kv_append_rotated(k, v, table, lens, **args)


@pytest.mark.parametrize("name", ["x", "freq", "norm"])
def test_backward_through_a_rotation_raises(tk, name):
    a = rotation()
    a[name].requires_grad_()
    q, _ = tk.kv_rotate(a["x"], None, a["pos"], a["freq"], q_norm=a["norm"])
    assert q.requires_grad
    with pytest.raises(RuntimeError, match="not implemented"):
        q.float().sum().backward()
    with pytest.raises(RuntimeError, match="no gradient"):
        tk.kv_rotate(a["x"], None, a["pos"], a["freq"], q_norm=a["norm"], q_out=torch.empty(3, 2, 64, dtype=F16).cuda())


def test_backward_through_the_frequencies_of_an_append_raises(tk):
    a = rotation()
    a["freq"].requires_grad_()
    with pytest.warns(UserWarning, match="freq"):
        q = appending(tk, a)
    with pytest.raises(RuntimeError, match="not implemented"):
        q.float().sum().backward()
    with pytest.warns(UserWarning, match="freq"):  # keys alone
        assert appending(tk, a, q=None, q_norm=None) is None
    with pytest.raises(RuntimeError, match="no gradient"):
        appending(tk, a, q_out=torch.empty(3, 2, 64, dtype=F16).cuda())
    with torch.no_grad(), warnings.catch_warnings():
        warnings.simplefilter("error")
        assert not appending(tk, a, q_out=torch.empty(3, 2, 64, dtype=F16).cuda()).requires_grad


@pytest.mark.parametrize("name", ["logits", "u", "temperature", "top_p", "min_p"])
def test_backward_through_a_sample_raises(tk, name):
    a = dict(logits=torch.randn(4, 100, device="cuda"), u=torch.full((4,), 0.5, device="cuda"),
             temperature=torch.ones(4, device="cuda"), top_p=torch.full((4,), 0.9, device="cuda"),
             min_p=torch.zeros(4, device="cuda"))
    a[name].requires_grad_()
    token, logp = tk.sample_rows(**a)
    assert logp.requires_grad and not token.requires_grad
    with pytest.raises(RuntimeError, match="not implemented"):
        logp.sum().backward()
    with pytest.raises(RuntimeError, match="no gradient"):
        tk.sample_rows(**a, logp=torch.zeros(4, device="cuda"))
    with torch.no_grad():
        assert not tk.sample_rows(**a, logp=torch.zeros(4, device="cuda"))[1].requires_grad


def test_tangents_are_refused(tk):
    """In forward mode too: nothing that comes back could have a tangent."""
    import torch.autograd.forward_ad as fwd

    a = rotation()
    x, q_out = a["x"], torch.empty(3, 2, 64, dtype=F16, device="cuda")
    s = dict(logits=torch.randn(4, 100, device="cuda"), u=torch.full((4,), 0.5, device="cuda"),
             temperature=torch.ones(4, device="cuda"), top_p=torch.full((4,), 0.9, device="cuda"),
             min_p=torch.zeros(4, device="cuda"), logp=torch.zeros(4, device="cuda"))
    with fwd.dual_level():
        def dual(t):
            return fwd.make_dual(t.detach().clone(), torch.ones_like(t))

        for kw in (dict(q=dual(x)), dict(k=dual(x)), dict(freq=dual(a["freq"])), dict(q_norm=dual(a["norm"])),
                   dict(k_norm=dual(a["norm"])), dict(q_out=dual(q_out))):
            args = dict(q=x, k=x, pos=a["pos"], freq=a["freq"], q_norm=a["norm"], k_norm=a["norm"])
            args.update(kw)
            with pytest.raises(NotImplementedError, match="forward mode"):
                tk.kv_rotate(**args)
        for kw in (dict(k_new=dual(x)), dict(v_new=dual(x)), dict(freq=dual(a["freq"])), dict(k_norm=dual(a["norm"])),
                   dict(q=dual(x)), dict(q_norm=dual(a["norm"])), dict(q_out=dual(q_out))):
            with pytest.raises(NotImplementedError, match="forward mode"):
                appending(tk, a, **kw)
        for name in s:
            with pytest.raises(NotImplementedError, match="forward mode"):
                tk.sample_rows(**{**s, name: dual(s[name])})
        # What has no tangent runs; so does everything where forward mode is off.
        tk.kv_rotate(x, x, a["pos"], a["freq"])
        both = dual(s["logits"])
        with torch.inference_mode():
            tk.sample_rows(**{**s, "logits": both})
        tk.sample_rows(**{**s, "logits": fwd.unpack_dual(both).primal})

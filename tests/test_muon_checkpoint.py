"""Checkpoints of MultiMuon: a list whose steps would be made of other coefficients,
eps, factors of the learning rate or updates' type is refused before anything is
written, and goes on bit for bit where they agree."""
from types import SimpleNamespace

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import zero_sharded_mixed_partition_amd as Z  # noqa: E402
from zero_sharded_mixed_partition_amd import checkpoint  # noqa: E402

SETTINGS = dict(coefs=[[3.4445, -4.775, 2.0315]] * 5, eps=1e-7, scales=[0.2 * 7 ** 0.5, 0.6], update_dtype="bfloat16")
OTHERS = dict(coefs=[[3.4445, -4.775, 2.0315]] * 4, eps=1e-8, scales=[1.0, 1.0], update_dtype="float16")


def opt(**settings):
    cols = [torch.full((n,), 1.0 + i) for i, n in enumerate((5, 7))]
    o = SimpleNamespace(state=None, t=0, scaler=Z.LossScaler(), hyper=[dict(lr=0.1)], cols=cols, groups=[0, 0],
                        checkpoint_arrays=lambda: {f"master_{i}": x for i, x in enumerate(cols)})
    if settings:
        o.checkpoint_settings = lambda: settings
    return o


@pytest.mark.parametrize("name", sorted(OTHERS))
def test_other_settings_are_refused(tmp_path, monkeypatch, name):
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(synchronize=lambda: None))
    saved = opt(**SETTINGS)
    for x in saved.cols:
        x.mul_(10)
    saved.t = 8
    checkpoint.save(saved, str(tmp_path))
    for other in (opt(**dict(SETTINGS, **{name: OTHERS[name]})), opt()):
        before = [x.clone() for x in other.cols]
        with pytest.raises(ValueError, match="written with other"):
            checkpoint.load(other, str(tmp_path))
        with pytest.raises(ValueError, match="written with other"):
            checkpoint.load_state_dict(other, checkpoint.state_dict(saved))
        assert other.t == 0 and all(torch.equal(x, y) for x, y in zip(before, other.cols))
    same = opt(**SETTINGS)
    checkpoint.load(same, str(tmp_path))
    assert same.t == 8 and all(torch.equal(x, y) for x, y in zip(saved.cols, same.cols))


def test_a_checkpoint_without_settings_still_loads(monkeypatch):
    """Earlier ones do not hold them."""
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(synchronize=lambda: None))
    d = checkpoint.state_dict(opt(**SETTINGS))
    del d["settings"]
    checkpoint.load_state_dict(opt(**SETTINGS), d)


@pytest.mark.gpu
def test_lists_on_the_device(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    rng = np.random.default_rng(0)
    shapes = [(48, 80), (130, 129)]

    def muon(**kw):
        ms = [torch.from_numpy(rng.normal(size=s).astype(np.float32)).cuda() for s in shapes]
        gs = [torch.from_numpy(rng.normal(size=s)).half().cuda() for s in shapes]
        return Z.MultiMuon(ms, gs, **kw), gs

    a, ga = muon(adjust="spectral", coefs=((1.5, -0.5, 0),) * 6, eps=1e-6)
    a.step()
    checkpoint.save(a, str(tmp_path))
    for kw in (dict(), dict(adjust="spectral"), dict(adjust="spectral", coefs=((1.5, -0.5, 0),) * 6),
               dict(adjust="rms", coefs=((1.5, -0.5, 0),) * 6, eps=1e-6),
               dict(adjust="spectral", coefs=((1.5, -0.5, 0),) * 6, eps=1e-6, update_dtype=torch.float16)):
        with pytest.raises(ValueError, match="written with other"):
            checkpoint.load(muon(**kw)[0], str(tmp_path))
    b, gb = muon(adjust="spectral", coefs=((1.5, -0.5, 0),) * 6, eps=1e-6)
    checkpoint.load(b, str(tmp_path))
    for x, y in zip(ga, gb):
        y.copy_(x)
    a.step()
    b.step()
    assert all(torch.equal(x, y) for x, y in zip(a.checkpoint_arrays().values(), b.checkpoint_arrays().values()))

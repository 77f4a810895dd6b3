"""Calls of the attention functions that lack a tensor they need: ValueError, before anything else is looked at."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def kvx():
    import kv_cache_attention_02_gb300 as k
    k.lib()
    return k


@pytest.mark.parametrize("lacks", ["q", "out", "k_new", "v_new"])
@pytest.mark.parametrize("name", ["attend_prompt", "attend_tree"])
def test_prompts_and_trees(kvx, name, lacks):
    q, x = torch.zeros(2, 5, 4, 64, dtype=torch.float16), torch.zeros(2, 5, 2, 64, dtype=torch.float16)
    given = dict(dict(q=q, out=q, k_new=x, v_new=x), **{lacks: None})
    with pytest.raises(ValueError, match="must be given"):
        getattr(kvx, name)(given.pop("q"), given.pop("out"), **given)


def test_joins(kvx, monkeypatch):
    x, lse = torch.zeros(5, 4, 64, dtype=torch.float16), torch.zeros(5, 4)
    for out, parts in ((None, [(x, lse)]), (x, None)):
        with pytest.raises(ValueError, match="must be given"):
            kvx.attend_join(out, parts)
    monkeypatch.setattr(kvx, "_place", lambda *a: (x.get_device(), 0))      # past the check of the device
    for part in ((None, lse), (x, None)):
        with pytest.raises(ValueError, match="part 1 must be given"):
            kvx.attend_join(x, [(x, lse), part])


def test_an_output_of_one_token(kvx, monkeypatch):
    monkeypatch.setattr(kvx, "_place", lambda *a: (-1, 0))
    q, k = torch.zeros(2, 4, 64, dtype=torch.float16), torch.zeros(2, 2, 5, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="out must be given"):
        kvx.attend(q, None, k=k, v=k)

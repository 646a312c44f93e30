"""Every form of kv4_evict's choice -- threads a CTA, CTAs a row, tokens a thread, scores held
or read again -- is run: which one a case takes is worked out from the dispatch in
csrc/kv4_evict.cu itself, so that a change of it cannot leave one untested."""
import os
import re

import numpy as np
import pytest

torch = pytest.importorskip("torch")
if torch.cuda.is_available():
    from kv4_inputs import ints
    from test_gpu_kv4_evict import bits, cache, expect, random_scores

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "nvfp4_gated_deltanet_gb300", "csrc",
                      "kv4_evict.cu")

# form: (KV heads, d, page_tokens, layers, [tokens], [kept], recent). Where a form is taken for many rows only, few
# tokens are kept of many and the rows are short of what the form holds.
CASES = {
    "256, 1, 4": (2, 64, 16, 1, [1000, 40, 0], [300, 40, 5], 8),
    "256, 1, 8": (1, 128, 64, 1, [2000, 1025], [700, 3], 0),
    "256, 1, 16": (1, 64, 64, 2, [3000, 4090], [100, 4000], 9),
    "512, 1, 16": (8, 64, 256, 20, [5000], [40], 4),
    "1024, 1, 16": (8, 64, 256, 20, [9000], [40], 4),
    "1024, 2, 16": (2, 64, 64, 40, [9000], [3], 1),
    "1024, 4, 16": (1, 64, 64, 2, [16001], [5000], 3),
    "1024, 8, 16": (1, 64, 64, 1, [30003, 17], [20011, 9], 3),
    "1024, 16, 16": (1, 64, 64, 1, [70000, 100], [300, 50], 10),
    "1024, 16, 0": (1, 64, 256, 1, [400000], [200], 10),
    "1024, 1, 0, false": (1, 64, 256, 1, [800000], [200], 10),
}


def dispatch():
    """form(most tokens of a row, rows) as launch_kv4_evict has it."""
    text = open(SOURCE).read()
    body = text[text.index("cudaError_t launch_kv4_evict"):]
    value = lambda name: eval(re.search(rf"constexpr int {name} = ([\d* ]+);", text).group(1))
    python = lambda c: c.replace("&&", " and ").replace("||", " or ").replace("/", "//")
    loop = python(re.search(r"while \((.*)\) cs \*= 2;", body).group(1))
    rules = re.findall(r"(?:if \(([^)]*)\)|else) e = launch_select<([^>]*)>", body)
    assert len(rules) > 1 and [c for c, _ in rules].count("") == 1 and rules[-1][0] == ""
    known = dict(kSplit=value("kSplit"), kMaxHeld=value("kMaxHeld"))

    def form(most, rows):
        cs = 1
        while eval(loop, known, dict(cs=cs, most=most, rows=rows)):
            cs *= 2
        here = dict(cs=cs, slice=(most + cs - 1) // cs)
        return next(f for c, f in rules if not c or eval(python(c), known, here))

    return form, [f for _, f in rules]


def test_every_form_has_a_case():
    form, forms = dispatch()
    assert sorted(forms) == sorted(CASES)
    for name, (hkv, d, page, layers, lens, keeps, recent) in CASES.items():
        cols = max(-(-n // page) for n in lens)
        assert form(min(max(lens), cols * page), layers * len(lens) * hkv) == name
    # of one CTA with orders in registers there are forms with as many bins as threads, fewer and more
    assert {"256, 1, 16", "512, 1, 16", "1024, 1, 16"} < set(forms)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["weights", "ties", "signs", "equal"])
@pytest.mark.parametrize("name", CASES)
def test_form(name, kind):
    """Exactly the plain choice and move, in place and to another tensor, ties and NaN at the border among them."""
    import nvfp4_gated_deltanet_gb300 as g
    hkv, d, page, layers, lens, keeps, recent = CASES[name]
    B, room, most = len(lens), max(lens), max(keeps)
    pages, tab, new = cache(lens, [min(k, n) for k, n in zip(keeps, lens)], page, hkv, d, layers, seed=B)
    scores = random_scores((layers, B, hkv, room), len(name), kind)
    want = expect(pages, tab, new, scores, list(range(B)), lens, keeps, recent, page, d, most)
    st = ints([0])
    other, copy = torch.full_like(scores, -5.0), pages.clone()
    kept, n = g.kv4_evict(copy, tab, ints(lens), ints(keeps), recent, scores, new, max_keep=most, scores_out=other, dev_status=st)
    assert np.array_equal(kept.cpu().numpy(), want[2]) and n.tolist() == [min(a, b) for a, b in zip(lens, keeps)]
    assert np.array_equal(copy.cpu().numpy(), want[0])
    for b, m in enumerate(lens):
        assert np.array_equal(bits(other[:, b, :, :m]), want[1][:, b, :, :m].view(np.int32)) and (other[:, b, :, m:] == -5).all()
    again, _ = g.kv4_evict(pages, tab, ints(lens), ints(keeps), recent, scores, new, max_keep=most, dev_status=st)
    assert torch.equal(again, kept) and torch.equal(pages, copy) and np.array_equal(bits(scores), want[1].view(np.int32))
    assert st.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", [n for n in CASES if n.split(", ")[1] == "1"])
@pytest.mark.parametrize("k,recent", [(0, 0), (1, 0), (1, 1), (2, 1)])
def test_few_kept(name, k, recent):
    """None, the best one, the newest one, one of each."""
    import nvfp4_gated_deltanet_gb300 as g
    hkv, d, page, layers, lens, _, _ = CASES[name]
    B, keeps = len(lens), [k] * len(lens)
    pages, tab, new = cache(lens, [max(k, 1)] * B, page, hkv, d, layers, seed=3)
    scores = random_scores((layers, B, hkv, max(lens)), 9, "signs")
    want = expect(pages, tab, new, scores, list(range(B)), lens, keeps, recent, page, d, max(k, 1))
    kept, _ = g.kv4_evict(pages, tab, ints(lens), ints(keeps), recent, scores, new, max_keep=max(k, 1))
    assert np.array_equal(kept.cpu().numpy(), want[2])
    assert np.array_equal(pages.cpu().numpy(), want[0]) and np.array_equal(bits(scores), want[1].view(np.int32))

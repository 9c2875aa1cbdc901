"""CPU checks of the rules that cut calls into work: the sizes that GPU tests run take the forms that they are there for."""
from tests import test_gated_forms_gpu as forms
from tests.plans import SMS, ask


def test_decode_cases_take_their_splits():
    plans = ask(*[("decode", m, n, k, SMS) for m, n, k, *_ in forms.DECODE])
    streams = ask(*[("streams", m, n, k, SMS) for m, n, k, *_ in forms.DECODE])
    for case, p, s in zip(forms.DECODE, plans, streams):
        kind = "none" if p["rest"] == 0 else "own" if p["rest_ctas"] % p["rest"] == 0 and p["rest_ctas"] > p["rest"] else "straddle"
        assert s["streams"] and (p["whole"], kind) == case[-2:], (case, p)

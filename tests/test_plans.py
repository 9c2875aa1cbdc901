"""CPU checks of the rules that cut calls into work: the sizes that GPU tests run take the forms that they are there for."""
from tests import test_fp8_forms_gpu as fp8
from tests import test_gated_forms_gpu as forms
from tests.plans import SMS, ask


def test_decode_cases_take_their_splits():
    plans = ask(*[("decode", m, n, k, SMS) for m, n, k, *_ in forms.DECODE])
    streams = ask(*[("streams", m, n, k, SMS) for m, n, k, *_ in forms.DECODE])
    for case, p, s in zip(forms.DECODE, plans, streams):
        kind = "none" if p["rest"] == 0 else "own" if p["rest_ctas"] % p["rest"] == 0 and p["rest_ctas"] > p["rest"] else "straddle"
        assert s["streams"] and (p["whole"], kind) == case[-2:], (case, p)


def test_two_mma_cases_take_two():
    for backward, cases in ((0, forms.TWO_MMAS_FWD), (1, forms.TWO_MMAS_DX)):
        plans = ask(*[("gemm", backward, m, n, k, r, SMS) for m, n, k, r, *_ in cases])
        assert all(p["parts"] == 2 for p in plans), plans
        # one of them ends with a token tile of a single part, one has more tiles than CTA pairs
        assert any(0 < m - (p["row_tiles"] - 1) * p["tile_rows"] <= 256 < p["tile_rows"] for (m, *_), p in zip(cases, plans))
        assert any(p["tiles"] > p["pairs"] for p in plans)


def test_split_cases_take_several_rounds():
    for (m, n, k, r, _), p in zip(forms.ROUNDS_OF_SPLITS, ask(*[("gemm", 0, m, n, k, r, SMS) for m, n, k, r, _ in forms.ROUNDS_OF_SPLITS])):
        assert p["splits"] > 1 and p["tiles"] > 2 * p["pairs"], ((m, n, k, r), p)


def test_streamed_8_bit_cases_take_several_rounds():
    for (m, n, k, *_, rounds), p in zip(fp8.STREAMED, ask(*[("fp8", m, n, k, SMS) for m, n, k, *_ in fp8.STREAMED])):
        assert p["streams"] and -(-p["groups"] // p["ctas"]) == rounds, ((m, n, k), p)

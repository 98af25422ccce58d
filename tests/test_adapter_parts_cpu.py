"""The inputs of adapter_parts.py tell three parts from two (a mistake planted in the oracle)."""
import adapter_parts as P


def test_two_parts_miss_the_bound_that_three_keep():
    for seed in range(3):
        c = P.case(seed=seed)
        want, three, two = P.results(c), P.results(c, 3), P.results(c, 2)
        for name in want:
            assert P.worst(three[name], want[name])[0] <= 2.0 ** -24 * 1.01, name      # h's and e's rounding alone
            top, share = P.worst(two[name], want[name])
            nonzero = float((want[name] != 0).double().mean())
            assert top > 4 * P.BOUND_ANY_ORDER and share > nonzero / 2, (name, top, share)

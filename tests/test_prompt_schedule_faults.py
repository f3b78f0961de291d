"""A fault that the prompt attention kernel once had, put back into its schedule model (tests/test_prompt_schedule.py):
a row tile without keys in an item does not take part in the barriers of its queries and outputs, so that their
phases are counted by the items in which it has keys; counted by all items, the parity names another phase.  And
the model's figures against the kernel's source."""
import inspect
import random
import re
import textwrap

import pytest

import test_prompt_schedule as schedule
from test_kernel_sources import block_at, source


def planted(old, new):
    """The model with one line of it changed."""
    src = textwrap.dedent(inspect.getsource(schedule.Cta))
    assert src.count(old) == 1
    space = dict(vars(schedule))
    exec(src.replace(old, new), space)
    return space["Cta"]


def faults(cta, D, n):
    rng, found = random.Random(D + 6), 0
    for _ in range(n):
        try:
            cta(schedule.random_items(rng, schedule.KINDS[D]["halves"]), rng=rng, **schedule.KINDS[D]).run()
        except schedule.Fault:
            found += 1
    return found


@pytest.mark.parametrize("D", [64, 128])
def test_the_model_finds_a_phase_counted_by_all_items(D):
    assert faults(planted("had += mine > 0", "had += 1"), D, 200) > 0
    assert faults(planted("had += mine > 0", "had += int(mine > 0)"), D, 200) == 0


def test_the_kernel_counts_them_by_items_with_keys():
    src = source("rkv_prompt_attention.cu")
    kernel = block_at(src, src.index("k_prompt_attention(const __grid_constant__"))
    assert "turns += mine > 0;" in kernel
    assert re.search(r"wait\(o_empty \+ h, turns \^ 1u\)", kernel) and re.search(r"q_full \+ h, turns\)", kernel)


def test_the_models_figures_are_the_kernels():
    cfg = block_at(source("rkv_prompt_attention.cu"), source("rkv_prompt_attention.cu").index("struct FlashCfg"))

    def value(name, D):
        expr = re.search(r"\b%s = ([^;,]*)[;,]" % name, cfg).group(1).replace("kTok", str(value("kTok", D)) if name != "kTok" else "")
        while "?" in expr:
            cond, rest = expr.split("?", 1)
            yes, no = rest.split(":", 1)
            expr = yes if eval(cond, {"D": D}) else no
        return eval(expr, {"D": D})

    for D, kind in schedule.KINDS.items():
        assert value("kHalves", D) == kind["halves"] and value("kBufs", D) == kind["bufs"] and value("kParts", D) == kind["parts"]
        assert value("kStages", D) == kind["stages"] and bool(value("kTurns", D)) == kind["turns"]
        assert bool(value("kQInTmem", D)) == kind.get("q_copied", False)

"""How the shared-prefix attention orders what one thread writes before another reads it, checked on its
source on the CPU: a run shows such a fault only where the schedule happens to."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "moe_decode_layer_mxfp8_gb300", "csrc")


def between(first, last):
    """The kernel's text from one place to the next occurrence of another, without comments."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "k_attend_shared.cu")).read())
    at = text.index(first) + len(first)
    return text[at:text.index(last, at)]


def test_an_items_fields_are_ordered_before_its_rows_are_made():
    """One lane writes the item, the whole warp reads it: a shuffle is no barrier for memory, a warp's
    barrier is."""
    steps = between("if (lane == 0) more = next_job(ar, plan, cur, job);", "item_rows(ar, plan, job)")
    assert "__syncwarp();" in steps


def test_streams_that_meet_order_what_they_read_of_each_others_tensor_memory():
    """The fence ahead of the arrival and the one behind the wait, whatever is read behind either meeting."""
    steps = between("auto meet = ", "};")
    at = [steps.index(x) for x in ("tc_fence_before();", "mbar_arrive(&ss.merge)", "wait(&ss.merge", "tc_fence_after();")]
    assert at == sorted(at)
    item = between("auto meet = ", "mbar_arrive(&ss.o_out[u])")
    assert item.count("meet()") == 2 and item.index("meet()") < item.index("ld_rows(") < item.rindex("meet()")

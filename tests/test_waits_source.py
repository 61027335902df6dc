"""Waits of whole warps in the FP8 projection's kernel for pairs, by reading its source: a wait that ran out is something
that no test may cause on purpose in that kernel. CPU only."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_sparse_attention_07_gb300", "csrc")


def function_body(text, name):
    """The text between the braces of a kernel."""
    at = text.index("{", text.index(name + "("))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i]
    raise AssertionError("no end")


def test_summing_warps_agree_on_a_wait_that_ran_out():
    """`ok` decides whether a warp takes part in the next vote, so all of its lanes have to have the same one: the summing
    warps wait by warp_wait alone."""
    with open(os.path.join(CSRC, "fp8_linear.cu"), encoding="utf-8") as f:
        body = function_body(f.read(), "fp8_linear_pair_kernel")
    body = re.sub(r"//[^\n]*", "", body)
    sums = body[body.index("regs_inc"):]
    assert len(re.findall(r"\bwarp_wait\w*(?:<\w+>)?\(", sums)) == 3 and not re.findall(r"\bmbar_wait", sums)
    # every wait of the control warps is one lane's (the copies) or the warp's (the products)
    control = body[body.index("regs_dec"):body.index("regs_inc")]
    copies, products = control.split("warp == 1 && half == 0")
    assert "lane == 0" in copies and not re.findall(r"\bmbar_wait", products)


def test_orders_between_the_ctas_of_a_cluster():
    """Waits on barriers that another CTA arrives on have the cluster's scope; a relaxed arrival at the cluster's barrier is
    made only where one warp arrives with release for the CTA's others, behind a barrier of theirs."""
    with open(os.path.join(CSRC, "fp8_linear.cu"), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    pair = function_body(text, "fp8_linear_pair_kernel")
    assert len(re.findall(r"\b(?:mbar|warp)_wait_cluster<(?:true|false)>\(", pair)) == 7
    assert not re.findall(r"\b(?:mbar|warp)_wait\(", pair) and "_relaxed(" not in pair.replace("mbar_arrive_relaxed(free0", "")
    # data behind copies and products: a fence for shared memory; hand-overs of tensor memory: tcgen05's fence behind the wait
    for bar in ("full(s)", "empty(s)", "got_bar"):
        assert re.findall(r"_wait_cluster<(\w+)>\(" + re.escape(bar), pair) in (["true"], ["true", "true"]), bar
    assert len(re.findall(r"acc_\w+\(.*\n?.*?tmem_fence_after", pair)) >= 2
    assert text.count("cluster_arrive_relaxed()") == 2           # its definition and
    join = function_body(text, "join_sums")
    assert re.search(r"bar\.arrive 2.*\n\s*cluster_arrive_relaxed\(\);", join)
    rows = function_body(text, "fp8_linear_rows_kernel")
    assert re.search(r"named_barrier\(2, kStore \+ 32\);\s*cluster_arrive\(\);", rows) and rows.rstrip().endswith("cluster_wait();")
    assert "cluster_meet" not in text

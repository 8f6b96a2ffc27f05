"""Source rules for the kernels' launch path (no GPU needed).

run() launches with programmatic stream serialisation, so a kernel launched
through it may be scheduled while the previous kernel in the stream is still
running.  Such a kernel must wait for its predecessor before it touches
memory: its first statement is pdl_enter().  A kernel that forgot it would
race with the kernel before it, so this is checked on the sources.
"""
import pathlib
import re

CSRC = pathlib.Path(__file__).resolve().parents[1] / "zero_partitioned_mixed_gb300" / "csrc"
LAUNCH = re.compile(r"\brun(?:_chunked(?:_u)?)?(?:<[^>(]*>)?\(\s*(k_\w+)")
KERNEL = re.compile(r"__global__ void (?:__launch_bounds__\([^)]*\) )?(k_\w+)\(([^)]*)\)\s*\{\n\s*([^\n]*)")


def _sources():
    return {p.name: p.read_text() for p in sorted(CSRC.glob("*.cu")) + sorted(CSRC.glob("*.cuh"))}


def test_kernels_launched_through_run_wait_for_their_predecessor():
    src = _sources()
    launched = {m.group(1) for t in src.values() for m in LAUNCH.finditer(t)}
    first = {}
    for t in src.values():
        for m in KERNEL.finditer(t):
            first.setdefault(m.group(1), []).append(m.group(3).strip())
    # the step, two-pass, fix-up, rollback, gather, reduce-scatter and ZeRO++ kernels
    assert {"k_step_spec", "k_gather", "k_rs", "k_fixup", "k_gather_q8", "k_rs_q"} <= launched
    for k in sorted(launched):
        assert k in first, f"{k} is launched through run() but its definition was not found"
        assert all(f == "pdl_enter();" for f in first[k]), f"{k} does not begin with pdl_enter(): {first[k]}"


def test_run_is_the_only_launch_with_the_attribute():
    # the attribute is set in one place; kernels launched with <<<>>> are plain
    src = _sources()
    hits = [n for n, t in src.items() if "cudaLaunchAttributeProgrammaticStreamSerialization" in t]
    assert hits == ["zero_device.cuh"]


def test_tensor_memory_is_allocated_before_the_next_kernel_may_start():
    # a block that let the next kernel's blocks in before its own allocation
    # could wait for tensor memory that they hold while they wait for it
    found = 0
    for name, t in _sources().items():
        for m in re.finditer(r"__global__ void[^{;]*?\b(k_\w+)\([^{;]*\)\s*\{(.*?)\n\}\n", t, re.S):
            body = m.group(2)
            alloc = re.search(r"\btmem_alloc(?:_pair)?\(", body)
            if not alloc:
                continue
            found += 1
            enter = body.find("pdl_enter();")
            if enter >= 0:
                assert alloc.start() < enter, f"{name}: {m.group(1)}"
                assert "__syncthreads();" in body[alloc.start():enter], f"{name}: {m.group(1)}"
    assert found >= 3


def test_no_block_with_tensor_memory_waits_for_blocks_that_may_wait_for_it():
    # Two clusters of different streams on the same two SMs: each has allocated on one of them and its second block
    # waits there behind the other's first.  Neither ends if a block keeps its tensor memory while it waits for its
    # cluster.  So a kernel frees it before it waits, or asks for so much shared memory that no other block with
    # tensor memory fits beside its own (the sizes are compared by static_assert).
    src = _sources()
    waiting = set()
    for name, t in src.items():
        for m in re.finditer(r"__global__ void[^{;]*?\b(k_\w+)\([^{;]*\)\s*\{(.*?)\n\}\n", t, re.S):
            body = m.group(2)
            alloc, free = (re.search(rf"\btmem_{w}(?:_pair)?\(", body) for w in ("alloc", "free"))
            if alloc and any(alloc.start() < s.start() < free.start() for s in re.finditer(r"\bcluster_sync\(\)", body)):
                waiting.add(m.group(1))
    assert waiting == {"k_ortho_small", "k_ortho_products"}
    assert re.search(r"if \(m\.ctas > 1 && smem < kAloneSmem\) smem = kAloneSmem;", src["zero_ortho.cu"])
    assert "static_assert(kProductSmem >= kAloneSmem" in src["zero_ortho.cu"]
    assert len(re.findall(r"static_assert\([^;]*>= kLeastTmemSmem", src["zero_mx4.cu"])) == 2


def test_a_block_asks_whether_a_wait_gave_up_after_its_barrier():
    # asked before it, the answer may come too early: another warp's wait can give up later, and the block would leave
    # (and free its tensor memory) with copies or products in flight
    found = 0
    for name, t in _sources().items():
        for m in re.finditer(r"__global__ void[^{;]*?\b(k_\w+)\([^{;]*\)\s*\{(.*?)\n\}\n", t, re.S):
            body = m.group(2)
            if "s_quit" not in body:
                continue
            found += 1
            free = re.search(r"\btmem_free(?:_pair)?\(", body).start()
            settle = body.rfind("settle(quit);", 0, free)
            barrier = body.rfind("__syncthreads();", 0, settle)
            assert 0 <= barrier < settle, f"{name}: {m.group(1)}"
            assert "bar_wait(" not in body[barrier:settle] and "finish()" not in body[barrier:settle], f"{name}: {m.group(1)}"
    assert found == 4


def test_waits_for_tensor_memory_loads_name_the_loaded_registers():
    # the registers of tcgen05.ld are filled only after tcgen05.wait::ld: a wait that does not name them lets the
    # compiler copy them before it
    t = _sources()["zero_tc.cuh"]
    loads = re.findall(r"void (\w+)\((?:uint32_t \w+, )?(?:uint32_t|float) \(&\w+\)\[(\d+)\]\) \{(.*?)\n\}\n", t, re.S)
    waits = [(name, int(n), body) for name, n, body in loads if "tcgen05.wait::ld" in body]
    assert sum(t.count(w) for w in ["tcgen05.wait::ld"]) == len(waits) == 2
    for name, n, body in waits:
        named = set(re.findall(r'"\+r"\(r\[(\d+)\]\)', body))
        assert named == {str(i) for i in range(n)}, name

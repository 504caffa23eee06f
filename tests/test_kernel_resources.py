"""Every kernel of libopq runs without scratch memory: the gfx950 assembly of
each HIP source, compiled with the library's flags (no GPU needed), reports no
private segment and no spilled vector register for any kernel."""
import re
from concurrent.futures import ThreadPoolExecutor

import pytest

from w4a16_linear_amd import build

HIP_SOURCES = [s for s in build.SOURCES if s.endswith(".hip")]


def _kernels(asm: str):
    """(name, {field: value}) for every kernel in the assembly's metadata."""
    meta = asm[asm.index("amdhsa.kernels:"):]
    for blk in re.split(r"\n  - \.", meta)[1:]:
        name = re.search(r"\.name:\s+(\S+)", blk)
        fields = {k: int(v) for k, v in re.findall(
            r"\.(private_segment_fixed_size|vgpr_spill_count|sgpr_spill_count|vgpr_count):\s+(\d+)", blk)}
        yield (name.group(1) if name else "?"), fields


@pytest.fixture(scope="module")
def assembly():
    with ThreadPoolExecutor(max_workers=len(HIP_SOURCES)) as ex:
        return dict(zip(HIP_SOURCES, ex.map(build.device_asm, HIP_SOURCES)))


@pytest.mark.slow
@pytest.mark.parametrize("src", HIP_SOURCES)
def test_no_scratch(assembly, src):
    kernels = list(_kernels(assembly[src]))
    assert kernels, f"no kernel metadata in {src}"
    bad = [(n, f) for n, f in kernels
           if f.get("private_segment_fixed_size", 0) or f.get("vgpr_spill_count", 0)]
    assert not bad, f"{src}: kernels using scratch: {bad[:3]}"


# ------------------------------------------------- waits behind matrix instructions

def _registers(text):
    """Vector registers named in operands: v5, v[4:7], a[0:3]."""
    out = set()
    for kind, first, last, one_kind, one in re.findall(r"\b([va])\[(\d+):(\d+)\]|\b([va])(\d+)\b", text):
        out |= {(one_kind, int(one))} if one else {(kind, r) for r in range(int(first), int(last) + 1)}
    return out


def _functions(asm):
    """{name: [(is label, text)]} of a listing's instructions and labels."""
    functions, code = {}, None
    for line in asm.splitlines():
        line = line.split(";")[0].strip()
        label = re.match(r"^(_ZN\S+|\.LBB\S+):$", line)
        if label and not line.startswith("."):
            code = functions.setdefault(label.group(1), [])
        elif line.startswith(".Lfunc_end"):
            code = None
        elif code is not None and line and (label or not line.startswith(".")):
            code.append((bool(label), label.group(1) if label else line))
    return functions


def _early_reads(code):
    """(wait states passed, matrix instruction, reader) where a matrix instruction's result is read too
    soon on some path.  The hardware does not wait: a reader has to be 8 wait states behind
    16x16x32 (four passes) and 12 behind 32x32x16 (eight), but for a matrix instruction that takes
    the result as the sum it adds to."""
    labels = {text: i for i, (is_label, text) in enumerate(code) if is_label}
    found = []
    for start, (is_label, text) in enumerate(code):
        if is_label or not text.startswith("v_mfma"):
            continue
        op, operands = text.split(None, 1)
        need = {"v_mfma_f32_16x16x32_bf16": 8, "v_mfma_f32_32x32x16_bf16": 12}[op]
        result = operands.split(",")[0]
        paths, seen = [(start + 1, 0, frozenset(_registers(result)))], set()
        while paths:
            at, waited, live = paths.pop()
            while at < len(code) and waited < need and live and (at, waited, live) not in seen:
                seen.add((at, waited, live))
                is_label, line = code[at]
                at += 1
                if is_label:
                    continue
                op, _, args = line.partition(" ")
                waited += int(args, 0) + 1 if op == "s_nop" else 1
                if op == "s_endpgm":
                    break
                if op == "s_branch":
                    at = labels.get(args.strip(), len(code))
                elif op.startswith("s_cbranch"):
                    if args.strip() in labels:
                        paths.append((labels[args.strip()], waited, live))
                elif not op.startswith("s_"):
                    first, _, rest = args.partition(",")
                    stores = op.startswith(("global_store", "buffer_store", "flat_store", "ds_write"))
                    if op.startswith("v_mfma") and rest.rpartition(",")[2].strip() == result:
                        rest = rest.rpartition(",")[0]
                    if _registers(args if stores else rest) & live:
                        found.append((waited - 1, text, line))
                    if not stores:
                        live = live - _registers(first)
    return found


def test_the_scan_for_early_reads():
    """On the copy of a sum that it was written for, and on what is right."""
    def listing(*between):
        return _functions("\n".join(("_ZN1fEv:", "v_mfma_f32_16x16x32_bf16 v[6:9], v[18:21], v[8:11], v[4:7]", *between,
                                     "s_endpgm", ".Lfunc_end0:")))["_ZN1fEv"]

    steps = ("s_add_i32 s5, s5, 1", "s_cmp_lt_i32 s5, s6", "v_add_u32_e32 v15, 1, v15", "s_cbranch_scc0 .LBB0_2")
    copy = ("v_mov_b64_e32 v[12:13], v[8:9]", ".LBB0_2:")
    assert [w for w, _, _ in _early_reads(listing(*steps, "s_nop 0", *copy))] == [5]
    assert not _early_reads(listing(*steps, "s_nop 3", *copy))
    assert [w for w, _, _ in _early_reads(listing("s_branch .LBB0_1", *steps, ".LBB0_1:", "global_store_dwordx2 v[0:1], v[6:7], off",
                                                  ".LBB0_2:"))] == [1]
    assert not _early_reads(listing("v_mfma_f32_16x16x32_bf16 v[10:13], v[18:21], v[22:25], v[6:9]", "s_nop 7"))
    assert len(_early_reads(listing("v_mfma_f32_16x16x32_bf16 v[10:13], v[6:9], v[22:25], v[6:9]", "s_nop 7"))) == 1
    assert not _early_reads(listing("v_mov_b32_e32 v6, v0", "v_mov_b32_e32 v1, v6", "s_nop 7"))   # a new value


@pytest.mark.slow
@pytest.mark.parametrize("src", HIP_SOURCES)
def test_matrix_results_are_waited_for(assembly, src):
    for name, code in _functions(assembly[src]).items():
        early = _early_reads(code)
        assert not early, f"{src}: {name}: {early[:3]}"

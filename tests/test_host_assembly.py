"""What the compiler made of the kernels, from the built objects: no vector
registers spilled and no scratch in the attention kernels, few scalars spilled,
and in no kernel a vector instruction between a place that waves skip to with an
empty mask and the mask's return there.

The last is a fault that the compiler (ROCm 7.2) has made where registers were
short and a loop's condition was a mask of lanes: copies of live values to other
registers stood before the mask's return, so that waves which had skipped the
branch lost them."""
import glob
import os
import re
import subprocess

import pytest

from tensor_compiler_tiling_amd import build as B

LLVM = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(B.HIPCC))), "llvm", "bin")
TARGET = f"hipv4-amdgcn-amd-amdhsa--{B.ARCH}"

# instructions that write a lane's registers or memory (reading a lane into a
# scalar, writing a lane by number and comparing do not depend on the mask so)
VECTOR = re.compile(r"(v_(?!readlane|readfirstlane|writelane|cmp|nop)|ds_|global_|flat_|buffer_|scratch_)")


def lost_copies(text: str) -> list[str]:
    """Kernels of a disassembly with a vector instruction between the target of a
    branch on an empty mask and the mask's return there."""
    lines = []  # (kernel, address, operation, operands)
    targets, kernel, base = set(), "", {}
    for line in text.splitlines():
        m = re.match(r"([0-9a-f]+) <(\S+)>:", line)
        if m:
            kernel = m.group(2)
            base[kernel] = int(m.group(1), 16)
            continue
        m = re.match(r"\s+(\S+)\s*(.*?)\s*// ([0-9A-F]+): [0-9A-F ]+(?:<(\S+?)(?:\+0x([0-9a-f]+))?>)?", line)
        if not m:
            continue
        op, args, address, symbol, offset = m.groups()
        lines.append((kernel, int(address, 16), op, args))
        if op == "s_cbranch_execz":
            targets.add(base[symbol] + int(offset or "0", 16))
    out, active, found = [], False, False
    for kernel, address, op, args in lines:
        if address in targets:
            active, found = True, False
        if not active:
            continue
        if op.startswith(("s_cbranch", "s_branch", "s_endpgm", "s_setpc", "s_and_saveexec")):
            active = False
        elif op in ("s_or_saveexec_b64", "s_andn2_saveexec_b64") or (op.startswith("s_") and args.startswith("exec")):
            if found:
                out.append(kernel)
            active = False
        elif VECTOR.match(op):
            found = True
    return out


def device_code(obj: str, tmp: str) -> str:
    fat, code = os.path.join(tmp, "fat"), os.path.join(tmp, "code")
    subprocess.run([f"{LLVM}/llvm-objcopy", "--dump-section", f".hip_fatbin={fat}", obj, os.devnull], check=True)
    subprocess.run([f"{LLVM}/clang-offload-bundler", "--type=o", "--unbundle", f"--input={fat}", f"--targets={TARGET}",
                    f"--output={code}"], check=True)
    return code


def objects() -> list[str]:
    objs = [os.path.join(B.BUILD, os.path.basename(k) + ".o") for k in sorted(glob.glob(os.path.join(B.CSRC, "*.hip")))]
    if not all(os.path.exists(o) for o in objs):
        B.build()
    return objs


@pytest.mark.parametrize("source", sorted(os.path.basename(k) for k in glob.glob(os.path.join(B.CSRC, "*.hip"))))
def test_no_copy_before_the_mask_returns(source, tmp_path):
    obj = next(o for o in objects() if os.path.basename(o) == source + ".o")
    code = device_code(obj, str(tmp_path))
    text = subprocess.run([f"{LLVM}/llvm-objdump", "-d", code], capture_output=True, text=True, check=True).stdout
    assert "s_endpgm" in text
    assert lost_copies(text) == []


def test_attention_has_its_registers(tmp_path):
    obj = next(o for o in objects() if os.path.basename(o) == "attention.hip.o")
    notes = subprocess.run([f"{LLVM}/llvm-readelf", "--notes", device_code(obj, str(tmp_path))], capture_output=True, text=True,
                           check=True).stdout
    kernels = re.findall(r"\.name: +(\S+kernel\S+)\n(?:.*\n)*?.*\.private_segment_fixed_size: (\d+)\n(?:.*\n)*?"
                         r".*\.sgpr_spill_count: (\d+)\n(?:.*\n)*?.*\.vgpr_spill_count: (\d+)", notes)
    assert len(kernels) == notes.count(".vgpr_spill_count") == 48
    for name, scratch, scalars, vectors in kernels:
        assert (int(scratch), int(vectors)) == (0, 0), name
        # strides and pointers that live through the whole kernel
        assert int(scalars) <= 64, (name, scalars)


SKIPPED = """
0000000000001000 <kernel_a>:
	s_and_saveexec_b64 s[2:3], vcc        // 000000001000: 00000000
	s_cbranch_execz 2                     // 000000001004: 00000000 <kernel_a+0x10>
	v_add_f32_e32 v1, v2, v3              // 000000001008: 00000000
	global_store_dword v[4:5], v1, off    // 00000000100C: 00000000
	{}
	s_or_b64 exec, exec, s[2:3]           // 000000001014: 00000000
	s_endpgm                              // 000000001018: 00000000
"""


@pytest.mark.parametrize("op,lost", [("v_accvgpr_write_b32 a3, v171", True), ("v_mov_b32_e32 v9, v8", True),
                                     ("ds_write_b32 v1, v2", True), ("s_nop 0", False), ("v_readlane_b32 s1, v9, 3", False)])
def test_the_search_finds_a_copy_that_is_lost(op, lost):
    text = SKIPPED.format(f"{op}   // 000000001010: 00000000")
    assert lost_copies(text) == (["kernel_a"] if lost else [])

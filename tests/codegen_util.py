"""A look at generated code for vector registers that are saved too late.

Where control flow joins, a block restores the lanes that took another way
(s_or_b64 exec, exec, ...).  A vector register that is saved to scratch memory, or copied to an
accumulator register, before that is saved for some of its lanes only, and what is
read back later is whatever lay there.  hipcc has made such code for a kernel that
spilled; a kernel that keeps its registers has nothing to save."""
import re

_KERNEL = re.compile(r"^(_Z\S+):")
_BLOCK = re.compile(r"^(\.LBB|; %bb)")
_RESTORE = re.compile(r"s_or_b64 exec, exec|s_(or|andn2)_saveexec_b64")
_NARROW = re.compile(r"s_(and|xor)_saveexec|s_\w+_b64 exec,")
_SAVE = re.compile(r"scratch_store|Folded Spill|accvgpr_write.*(Spill|Reload Reuse)")


def saved_before_restore(asm):
    """(kernel, instruction) of each register saved in a block ahead of the
    restore that the block begins with."""
    found, kernel, pending = [], None, []
    for line in asm.splitlines():
        m = _KERNEL.match(line)
        if m:
            kernel = m.group(1)
        if m or _BLOCK.match(line):
            pending = []                     # None: past the block's beginning
        elif pending is not None:
            if _RESTORE.search(line):
                found += [(kernel, x) for x in pending]
                pending = None
            elif _NARROW.search(line):
                pending = None
            elif _SAVE.search(line):
                pending.append(line.strip())
    return found

"""Writes acc_pinned.h, pinned_stage.inc, acc_scaled.h and scaled_stage.inc beside this script.

The 4-wave 256-tile product keeps each wave's 128 x 128 accumulator tile in
the AGPRs a0..a255, block (i, j) of its 8 x 8 blocks of 16 x 16 in
a[4 (8 i + j)] .. + 3. Every MFMA that updates a block names those registers in
inline asm, so the accumulators stay in place across the K loop (left to the
register allocator, a tile of this size is moved between registers inside the
loop). pinned_stage.inc is the unrolled schedule of one K stage (two k-groups of
32): MFMAs in pairs, with the fragment reads, operand loads and the stage
barrier spread between the pairs.

acc_scaled.h has the 8-bit products' MFMA for the same registers (one instruction
for a block's 128 k, with both operands' scales), and scaled_stage.inc their K
stage: the A fragments pass through four registers sets, the next stage's B
fragments are read meanwhile.

Run: python3 gen_acc_pinned.py  (the outputs are committed).
"""
import os

HERE = os.path.dirname(os.path.abspath(__file__))


def reg(q):
    return 4 * q


def header():
    out = ["// Generated by gen_acc_pinned.py: do not edit by hand.",
           "// Accumulators of the 4-wave 256-tile product in the AGPRs a0..a255: block",
           "// q = 8 i + j (i, j < 8) of a wave's 8 x 8 blocks of 16 x 16 in a[4 q] .. a[4 q + 3].",
           "// Included by ns_kernels.hip inside its namespace, after the bf16x8 and f32x4",
           "// typedefs and <type_traits>.",
           "#pragma once", "",
           "namespace pinned {", ""]
    # zero
    for part in range(8):
        body = " ".join(f'"v_accvgpr_write_b32 a{32 * part + k}, 0\\n"' for k in range(32))
        clob = ", ".join(f'"a{32 * part + k}"' for k in range(32))
        out.append(f"__device__ __forceinline__ void zero{part}() {{ asm volatile({body} ::: {clob}); }}")
    out.append("// Every accumulator to +0, then wait states before the first MFMA reads them.")
    out.append("__device__ __forceinline__ void zero() {")
    out.append("    zero0(); zero1(); zero2(); zero3(); zero4(); zero5(); zero6(); zero7();")
    out.append('    asm volatile("s_nop 7\\n s_nop 7");')
    out.append("}")
    out.append("")
    # mfma, read, write per block
    for q in range(64):
        r = reg(q)
        out.append(f"__device__ __forceinline__ void mfma{q}(bf16x8 a, bf16x8 b) {{")
        out.append(f'    asm volatile("v_mfma_f32_16x16x32_bf16 a[{r}:{r + 3}], %0, %1, a[{r}:{r + 3}]"')
        out.append(f'                 :: "v"(a), "v"(b) : "a{r}", "a{r + 1}", "a{r + 2}", "a{r + 3}");')
        out.append("}")
    for q in range(64):
        r = reg(q)
        out.append(f"__device__ __forceinline__ f32x4 rd{q}() {{")
        out.append("    f32x4 v;")
        out.append(f'    asm volatile("v_accvgpr_read_b32 %0, a{r}\\n v_accvgpr_read_b32 %1, a{r + 1}\\n"')
        out.append(f'                 "v_accvgpr_read_b32 %2, a{r + 2}\\n v_accvgpr_read_b32 %3, a{r + 3}"')
        out.append('                 : "=v"(v[0]), "=v"(v[1]), "=v"(v[2]), "=v"(v[3]));')
        out.append("    return v;")
        out.append("}")
    for q in range(64):
        r = reg(q)
        out.append(f"__device__ __forceinline__ void wr{q}(f32x4 v) {{")
        out.append(f'    asm volatile("v_accvgpr_write_b32 a{r}, %0\\n v_accvgpr_write_b32 a{r + 1}, %1\\n"')
        out.append(f'                 "v_accvgpr_write_b32 a{r + 2}, %2\\n v_accvgpr_write_b32 a{r + 3}, %3"')
        out.append(f'                 :: "v"(v[0]), "v"(v[1]), "v"(v[2]), "v"(v[3]) : "a{r}", "a{r + 1}", "a{r + 2}", "a{r + 3}");')
        out.append("}")
    out.append("")
    out.append("// Wait states between the last MFMA and the first read of its accumulators.")
    out.append('__device__ __forceinline__ void drain() { asm volatile("s_nop 7\\n s_nop 7\\n s_nop 7" ::: "memory"); }')
    out.append("")
    out.append("// f(std::integral_constant<int, q>, block q's four values) for every block, in order.")
    out.append("template <class F> __device__ __forceinline__ void each_block(F &&f) {")
    for q in range(64):
        out.append(f"    f(std::integral_constant<int, {q}>{{}}, rd{q}());")
    out.append("}")
    out.append("")
    out.append("// Block q = f(std::integral_constant<int, q>) for every block, then wait states")
    out.append("// before MFMAs read them.")
    out.append("template <class F> __device__ __forceinline__ void init_each_block(F &&f) {")
    for q in range(64):
        out.append(f"    wr{q}(f(std::integral_constant<int, {q}>{{}}));")
    out.append('    asm volatile("s_nop 7\\n s_nop 7");')
    out.append("}")
    out.append("")
    out += ["}  // namespace pinned", ""]
    return "\n".join(out)


def stage():
    # fragments: x < 8 the P (A operand) blocks, x >= 8 the Q (B operand) blocks; B first
    def fx(n):
        return 8 + n if n < 8 else n - 8
    G = 2
    ngrp = 64 // G
    body = ["// Generated by gen_acc_pinned.py: one K stage of the 4-wave 256-tile product.",
            "// In scope: F[2][16] fragments (slot 0 holds k-group 0's), rf(slot, buf, kg, x),",
            "// ld(n, kb, buf) (operand load n < 16 of stage kb into buffer buf), PAR (this",
            "// stage's buffer), kb, W (a next stage exists), L (stage kb + 2 exists)."]
    ops0 = [f"rf(1, PAR, 1, {fx(n)});" for n in range(16)]
    per0 = [ops0[k * 16 // ngrp:(k + 1) * 16 // ngrp] for k in range(ngrp)]
    for k in range(ngrp):
        for q in range(k * G, (k + 1) * G):
            body.append(f"pinned::mfma{q}(F[0][{q >> 3}], F[0][{8 + (q & 7)}]);")
        body += per0[k]
    ops1 = []
    for n in range(16):
        ops1.append(f"if (L) ld({n}, kb + 2, PAR);")
        ops1.append(f"if (W) rf(0, PAR ^ 1, 0, {fx(n)});")
    rest = ngrp - 1
    per1 = [ops1[k * len(ops1) // rest:(k + 1) * len(ops1) // rest] for k in range(rest)]
    for k in range(ngrp):
        for q in range(k * G, (k + 1) * G):
            body.append(f"pinned::mfma{q}(F[1][{q >> 3}], F[1][{8 + (q & 7)}]);")
        if k == 0:
            body.append("if (W) {")
            body.append("    wait_vmcnt<0>();   // this wave's loads of stage kb + 1")
            body.append("    lds_barrier();     // ... and every wave's; stage kb's buffer is read")
            body.append("}")
        else:
            body += per1[k - 1]
    return "\n".join(body) + "\n"


def scaled_header():
    out = ["// Generated by gen_acc_pinned.py: do not edit by hand.",
           "// The 8-bit products' MFMA on block q of the accumulators of acc_pinned.h: a's and b's",
           "// scales are the low bytes of sa and sb. Included by scaled.hip inside its namespace.",
           "#pragma once", "", "namespace pinned {", ""]
    for q in range(64):
        r = reg(q)
        out.append(f"__device__ __forceinline__ void scaled{q}(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {{")
        out.append(f'    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[{r}:{r + 3}], %0, %1, a[{r}:{r + 3}], %2, %3 op_sel_hi:[0,0,0]"')
        out.append(f'                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a{r}", "a{r + 1}", "a{r + 2}", "a{r + 3}");')
        out.append("}")
    out += ["", "}  // namespace pinned", ""]
    return "\n".join(out)


def scaled_stage():
    body = ["// Generated by gen_acc_pinned.py: one K stage of the 8-bit 256-tile product.",
            "// In scope: FA[4], FB[2][8] fragments (FA[0] .. FA[2] and FB[PAR] hold this stage's),",
            "// ra(slot, i), rb(slot, j) (read a fragment of this stage's A, of the next stage's B),",
            "// rna(slot, i) (of the next stage's A), la(n), lb(n) (loads n < 8 of the A and the B panel",
            "// three stages on; n < 4 of A: the first halves of both wave rows), sa[8], sb(j), PAR."]
    slots = [[] for _ in range(64)]   # the operations after each MFMA
    slots[17].append("lds_barrier();     // every wave has the next stage's B")
    slots[47] += ["wait_vmcnt<16>();  // this wave's loads of the next A panel and the B panel after the next",
                  "lds_barrier();     // ... and every wave's; this stage's A is read"]
    for i, k in enumerate((1, 9, 17, 25, 33)):      # as soon as the slot's last fragment has been used
        slots[k].append(f"ra({(i + 3) & 3}, {i + 3});")
    for n, k in enumerate((49, 51, 57)):
        slots[k].append(f"rna({n}, {n});")
    for n, k in enumerate((1, 3, 3, 5, 5, 7, 7, 9)):
        slots[k].append(f"rb(PAR ^ 1, {n});")
    for n, k in enumerate((17, 19, 21, 23, 27, 29, 31, 35)):
        slots[k].append(f"lb({n});")
    for n, k in enumerate((49, 51, 53, 55, 57, 59, 61, 63)):
        slots[k].append(f"la({n});")
    for q in range(64):
        i, j = q >> 3, q & 7
        body.append(f"pinned::scaled{q}(FB[PAR][{j}], FA[{i & 3}], sb({j}), sa[{i}]);")
        body += slots[q]
    return "\n".join(body) + "\n"


if __name__ == "__main__":
    with open(os.path.join(HERE, "acc_pinned.h"), "w") as f:
        f.write(header())
    with open(os.path.join(HERE, "pinned_stage.inc"), "w") as f:
        f.write(stage())
    with open(os.path.join(HERE, "acc_scaled.h"), "w") as f:
        f.write(scaled_header())
    with open(os.path.join(HERE, "scaled_stage.inc"), "w") as f:
        f.write(scaled_stage())
    print("wrote acc_pinned.h, pinned_stage.inc, acc_scaled.h, scaled_stage.inc")

// Generated by gen_acc_pinned.py: do not edit by hand.
// The 8-bit products' MFMA on block q of the accumulators of acc_pinned.h: a's and b's
// scales are the low bytes of sa and sb. Included by scaled.hip inside its namespace.
#pragma once

namespace pinned {

__device__ __forceinline__ void scaled0(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[0:3], %0, %1, a[0:3], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a0", "a1", "a2", "a3");
}
__device__ __forceinline__ void scaled1(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[4:7], %0, %1, a[4:7], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a4", "a5", "a6", "a7");
}
__device__ __forceinline__ void scaled2(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[8:11], %0, %1, a[8:11], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a8", "a9", "a10", "a11");
}
__device__ __forceinline__ void scaled3(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[12:15], %0, %1, a[12:15], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a12", "a13", "a14", "a15");
}
__device__ __forceinline__ void scaled4(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[16:19], %0, %1, a[16:19], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a16", "a17", "a18", "a19");
}
__device__ __forceinline__ void scaled5(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[20:23], %0, %1, a[20:23], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a20", "a21", "a22", "a23");
}
__device__ __forceinline__ void scaled6(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[24:27], %0, %1, a[24:27], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a24", "a25", "a26", "a27");
}
__device__ __forceinline__ void scaled7(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[28:31], %0, %1, a[28:31], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a28", "a29", "a30", "a31");
}
__device__ __forceinline__ void scaled8(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[32:35], %0, %1, a[32:35], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a32", "a33", "a34", "a35");
}
__device__ __forceinline__ void scaled9(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[36:39], %0, %1, a[36:39], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a36", "a37", "a38", "a39");
}
__device__ __forceinline__ void scaled10(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[40:43], %0, %1, a[40:43], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a40", "a41", "a42", "a43");
}
__device__ __forceinline__ void scaled11(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[44:47], %0, %1, a[44:47], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a44", "a45", "a46", "a47");
}
__device__ __forceinline__ void scaled12(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[48:51], %0, %1, a[48:51], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a48", "a49", "a50", "a51");
}
__device__ __forceinline__ void scaled13(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[52:55], %0, %1, a[52:55], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a52", "a53", "a54", "a55");
}
__device__ __forceinline__ void scaled14(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[56:59], %0, %1, a[56:59], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a56", "a57", "a58", "a59");
}
__device__ __forceinline__ void scaled15(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[60:63], %0, %1, a[60:63], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a60", "a61", "a62", "a63");
}
__device__ __forceinline__ void scaled16(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[64:67], %0, %1, a[64:67], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a64", "a65", "a66", "a67");
}
__device__ __forceinline__ void scaled17(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[68:71], %0, %1, a[68:71], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a68", "a69", "a70", "a71");
}
__device__ __forceinline__ void scaled18(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[72:75], %0, %1, a[72:75], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a72", "a73", "a74", "a75");
}
__device__ __forceinline__ void scaled19(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[76:79], %0, %1, a[76:79], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a76", "a77", "a78", "a79");
}
__device__ __forceinline__ void scaled20(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[80:83], %0, %1, a[80:83], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a80", "a81", "a82", "a83");
}
__device__ __forceinline__ void scaled21(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[84:87], %0, %1, a[84:87], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a84", "a85", "a86", "a87");
}
__device__ __forceinline__ void scaled22(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[88:91], %0, %1, a[88:91], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a88", "a89", "a90", "a91");
}
__device__ __forceinline__ void scaled23(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[92:95], %0, %1, a[92:95], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a92", "a93", "a94", "a95");
}
__device__ __forceinline__ void scaled24(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[96:99], %0, %1, a[96:99], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a96", "a97", "a98", "a99");
}
__device__ __forceinline__ void scaled25(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[100:103], %0, %1, a[100:103], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a100", "a101", "a102", "a103");
}
__device__ __forceinline__ void scaled26(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[104:107], %0, %1, a[104:107], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a104", "a105", "a106", "a107");
}
__device__ __forceinline__ void scaled27(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[108:111], %0, %1, a[108:111], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a108", "a109", "a110", "a111");
}
__device__ __forceinline__ void scaled28(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[112:115], %0, %1, a[112:115], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a112", "a113", "a114", "a115");
}
__device__ __forceinline__ void scaled29(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[116:119], %0, %1, a[116:119], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a116", "a117", "a118", "a119");
}
__device__ __forceinline__ void scaled30(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[120:123], %0, %1, a[120:123], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a120", "a121", "a122", "a123");
}
__device__ __forceinline__ void scaled31(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[124:127], %0, %1, a[124:127], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a124", "a125", "a126", "a127");
}
__device__ __forceinline__ void scaled32(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[128:131], %0, %1, a[128:131], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a128", "a129", "a130", "a131");
}
__device__ __forceinline__ void scaled33(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[132:135], %0, %1, a[132:135], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a132", "a133", "a134", "a135");
}
__device__ __forceinline__ void scaled34(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[136:139], %0, %1, a[136:139], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a136", "a137", "a138", "a139");
}
__device__ __forceinline__ void scaled35(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[140:143], %0, %1, a[140:143], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a140", "a141", "a142", "a143");
}
__device__ __forceinline__ void scaled36(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[144:147], %0, %1, a[144:147], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a144", "a145", "a146", "a147");
}
__device__ __forceinline__ void scaled37(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[148:151], %0, %1, a[148:151], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a148", "a149", "a150", "a151");
}
__device__ __forceinline__ void scaled38(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[152:155], %0, %1, a[152:155], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a152", "a153", "a154", "a155");
}
__device__ __forceinline__ void scaled39(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[156:159], %0, %1, a[156:159], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a156", "a157", "a158", "a159");
}
__device__ __forceinline__ void scaled40(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[160:163], %0, %1, a[160:163], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a160", "a161", "a162", "a163");
}
__device__ __forceinline__ void scaled41(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[164:167], %0, %1, a[164:167], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a164", "a165", "a166", "a167");
}
__device__ __forceinline__ void scaled42(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[168:171], %0, %1, a[168:171], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a168", "a169", "a170", "a171");
}
__device__ __forceinline__ void scaled43(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[172:175], %0, %1, a[172:175], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a172", "a173", "a174", "a175");
}
__device__ __forceinline__ void scaled44(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[176:179], %0, %1, a[176:179], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a176", "a177", "a178", "a179");
}
__device__ __forceinline__ void scaled45(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[180:183], %0, %1, a[180:183], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a180", "a181", "a182", "a183");
}
__device__ __forceinline__ void scaled46(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[184:187], %0, %1, a[184:187], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a184", "a185", "a186", "a187");
}
__device__ __forceinline__ void scaled47(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[188:191], %0, %1, a[188:191], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a188", "a189", "a190", "a191");
}
__device__ __forceinline__ void scaled48(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[192:195], %0, %1, a[192:195], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a192", "a193", "a194", "a195");
}
__device__ __forceinline__ void scaled49(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[196:199], %0, %1, a[196:199], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a196", "a197", "a198", "a199");
}
__device__ __forceinline__ void scaled50(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[200:203], %0, %1, a[200:203], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a200", "a201", "a202", "a203");
}
__device__ __forceinline__ void scaled51(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[204:207], %0, %1, a[204:207], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a204", "a205", "a206", "a207");
}
__device__ __forceinline__ void scaled52(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[208:211], %0, %1, a[208:211], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a208", "a209", "a210", "a211");
}
__device__ __forceinline__ void scaled53(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[212:215], %0, %1, a[212:215], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a212", "a213", "a214", "a215");
}
__device__ __forceinline__ void scaled54(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[216:219], %0, %1, a[216:219], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a216", "a217", "a218", "a219");
}
__device__ __forceinline__ void scaled55(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[220:223], %0, %1, a[220:223], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a220", "a221", "a222", "a223");
}
__device__ __forceinline__ void scaled56(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[224:227], %0, %1, a[224:227], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a224", "a225", "a226", "a227");
}
__device__ __forceinline__ void scaled57(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[228:231], %0, %1, a[228:231], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a228", "a229", "a230", "a231");
}
__device__ __forceinline__ void scaled58(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[232:235], %0, %1, a[232:235], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a232", "a233", "a234", "a235");
}
__device__ __forceinline__ void scaled59(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[236:239], %0, %1, a[236:239], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a236", "a237", "a238", "a239");
}
__device__ __forceinline__ void scaled60(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[240:243], %0, %1, a[240:243], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a240", "a241", "a242", "a243");
}
__device__ __forceinline__ void scaled61(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[244:247], %0, %1, a[244:247], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a244", "a245", "a246", "a247");
}
__device__ __forceinline__ void scaled62(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[248:251], %0, %1, a[248:251], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a248", "a249", "a250", "a251");
}
__device__ __forceinline__ void scaled63(i32x8 a, i32x8 b, uint32_t sa, uint32_t sb) {
    asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 a[252:255], %0, %1, a[252:255], %2, %3 op_sel_hi:[0,0,0]"
                 :: "v"(a), "v"(b), "v"(sa), "v"(sb) : "a252", "a253", "a254", "a255");
}

}  // namespace pinned

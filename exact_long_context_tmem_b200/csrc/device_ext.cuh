// What the tree decode and the cache's upkeep use beyond ptx.cuh and status.cuh (which the measured traffic
// of the other kernels is recorded against): bad arguments met on the device, shared memory by address,
// dependent launches and a few more instructions.
#pragma once

#include "ptx.cuh"

namespace attn {

// ---------------------------------------------------------------- status

// After DeviceErrorCode: an index or length among the arguments on the device is out of range.
static constexpr uint32_t ATTN_DEV_BAD_INDEX = 3;

// After WaitSite.
enum ArgSite : int {
  SITE_TR_LOAD = 50,
  SITE_TR_MMA_Q = 51,
  SITE_TR_MMA_U = 52,
  SITE_TR_MMA_P = 53,
  SITE_TR_CONV = 54,
  SITE_TR_SM_S = 55,
  SITE_TR_SM_SC = 56,
  SITE_TR_SM_V = 57,
  SITE_TR_EPI = 58,
  SITE_TR_DRAIN = 59,
  SITE_TR_PAGE = 60,
  SITE_TR_SCALE = 61,
  SITE_ACCEPT = 70,
  SITE_PAGES_COPY = 71,
  SITE_PAGES_COMPACT = 72,
  SITE_PAGES_FORK = 73,
};

// (code << 16) | site of the first bad argument since the last reset.  A word of its own: waits give up when
// g_dev_status is set, and an index that was skipped is no reason for other work to stop.
__device__ uint32_t g_arg_status = 0;

__device__ __forceinline__ void record_arg_error(uint32_t code, int site) {
  atomicCAS(&g_arg_status, 0u, (code << 16) | (uint32_t)(site & 0xFFFF));
}

// ---------------------------------------------------------------- shared memory by address

// 4 or 16 bytes from a shared-memory address.
__device__ __forceinline__ float lds_f1(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ float4 lds_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ uint4 lds_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds_u2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts_u4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
               : "memory");
}

// ---------------------------------------------------------------- dependent launches

// In a kernel launched as the dependent of another (launch_dependent on the host): waits for that one to have
// finished, its writes visible.  In the other: lets the dependent start its CTAs where there is room.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---------------------------------------------------------------- TMA, TMEM, packed fp32

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3, int c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\t mov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 d, a, b;\n\t mov.b64 {%0, %1}, d;}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

}  // namespace attn

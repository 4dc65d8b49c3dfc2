// Host side of the C ABI declared in include/ckda.h: argument validation,
// shape dispatch and error reporting.  Validation never touches the GPU, so a
// non-OK status means nothing was enqueued; only a launch can return
// CKDA_ERR_HIP.
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <string>

#include "ckda_internal.h"

namespace {

thread_local std::string g_last_error;

ckda_status_t fail(ckda_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
ckda_status_t fail(ckda_status_t s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return s;
}

ckda_status_t ok() {
  g_last_error.clear();
  return CKDA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range {
  const char* name;
  uintptr_t lo, hi;  // [lo, hi)
};

Range range(const char* name, const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{name, lo, lo + static_cast<uintptr_t>(bytes)};
}

bool overlap(const Range& a, const Range& b) {
  return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo;
}

int64_t elem_bytes(int32_t dtype) { return dtype == CKDA_DTYPE_BF16 ? 2 : 4; }

static_assert(CKDA_GATES_F32 == 0 && CKDA_GATES_LOGITS_F32 == 1 && CKDA_GATES_LOGITS_BF16 == 2,
              "the kernels index their variants by ckda_gate_input_t");
// q/k heads: 0 means as many as value heads
int32_t qk_heads_of(int32_t H, int32_t qk_heads) { return qk_heads == 0 ? H : qk_heads; }
bool valid_qk_heads(int32_t H, int32_t qk_heads) {
  const int32_t hk = qk_heads_of(H, qk_heads);
  return hk > 0 && H > 0 && H % hk == 0;
}

bool valid_gate_input(int32_t g) { return g >= CKDA_GATES_F32 && g <= CKDA_GATES_LOGITS_BF16; }
int64_t gate_bytes(int32_t g) { return g == CKDA_GATES_LOGITS_BF16 ? 2 : 4; }

ckda_status_t from_hip(hipError_t e) {
  if (e == hipSuccess) return ok();
  return fail(CKDA_ERR_HIP, "HIP launch error %d: %s", static_cast<int>(e), hipGetErrorString(e));
}

// ---- static scratch of ckda_chunk_fwd_noalloc
// Device memory the allocation-free forward uses as its workspace: every GPU
// the library runs on holds its own copy for the life of the process.  In
// host code `scratch` names a host-side stand-in, never a device address:
// its device address comes from hipGetSymbolAddress, once per device with
// that device current, and only that address is handed to kernels.
__device__ __align__(256) unsigned char scratch[CKDA_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mutex;
void* g_scratch_ptr[kMaxDevices];  // per device; nullptr until looked up

// The device address of the scratch copy on the device that `stream` belongs
// to (the current device for the null stream).
hipError_t scratch_address(hipStream_t stream, void** out) {
  int cur = -1;
  hipError_t e = hipGetDevice(&cur);
  if (e != hipSuccess) return e;
  int dev = cur;
  if (stream != nullptr) {
    e = hipStreamGetDevice(stream, &dev);
    if (e != hipSuccess) return e;
  }
  if (dev < 0 || dev >= kMaxDevices) return hipErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(g_scratch_mutex);
  if (g_scratch_ptr[dev] == nullptr) {
    if (dev != cur && (e = hipSetDevice(dev)) != hipSuccess) return e;
    void* p = nullptr;
    e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
    if (dev != cur) {
      const hipError_t r = hipSetDevice(cur);
      if (e == hipSuccess) e = r;
    }
    if (e != hipSuccess) return e;
    if (p == nullptr) return hipErrorInvalidSymbol;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return hipSuccess;
}

}  // namespace

extern "C" {

int32_t ckda_abi_version(void) { return CKDA_ABI_VERSION; }

const char* ckda_last_error(void) { return g_last_error.c_str(); }

const char* ckda_status_string(int32_t s) {
  switch (s) {
    case CKDA_OK: return "ok";
    case CKDA_ERR_INVALID_ARGUMENT: return "invalid argument";
    case CKDA_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case CKDA_ERR_WORKSPACE_TOO_SMALL: return "workspace too small";
    case CKDA_ERR_HIP: return "HIP runtime error";
  }
  return "unknown status";
}

int32_t ckda_fwd_supported(const ckda_fwd_desc_t* d) {
  if (!d) return 0;
  return ckda::fwd_supported(d->chunk_size, d->dk, d->dv, d->io_dtype) ? 1 : 0;
}

size_t ckda_chunk_fwd_workspace_size(const ckda_fwd_desc_t* d, int32_t packed) {
  if (!d || d->B <= 0 || d->T < 0 || d->H <= 0 || d->dk <= 0 || d->num_seqs < 0) return 0;
  if (d->io_dtype != CKDA_DTYPE_BF16 && d->io_dtype != CKDA_DTYPE_F32) return 0;
  if (d->chunk_size != 16 && d->chunk_size != 32 && d->chunk_size != 64) return 0;
  if (static_cast<int64_t>(d->B) * d->T == 0 || d->num_seqs == 0) return 0;
  return ckda::fwd_workspace_bytes(d->B, d->T, d->H, d->dk, d->num_seqs, d->chunk_size,
                                   d->io_dtype, packed != 0, d->sign_absorb == 1);
}

size_t ckda_chunk_bwd_workspace_size(const ckda_fwd_desc_t* d, int32_t packed) {
  if (!d || d->B <= 0 || d->T < 0 || d->H <= 0 || d->dk <= 0 || d->dv <= 0 || d->num_seqs < 0)
    return 0;
  if (d->io_dtype != CKDA_DTYPE_BF16 && d->io_dtype != CKDA_DTYPE_F32) return 0;
  if (d->chunk_size != 16 && d->chunk_size != 32 && d->chunk_size != 64) return 0;
  if (static_cast<int64_t>(d->B) * d->T == 0 || d->num_seqs == 0) return 0;
  if (!valid_gate_input(d->gate_input) || !valid_qk_heads(d->H, d->qk_heads)) return 0;
  const size_t core = ckda::bwd_workspace_bytes(d->B, d->T, d->H, d->dk, d->dv, d->num_seqs,
                                                d->chunk_size, d->io_dtype, packed != 0);
  const size_t extra = ckda::bwd_gates_extra_bytes(d->B, d->T, d->H, qk_heads_of(d->H, d->qk_heads),
                                                   d->dk, d->io_dtype, d->gate_input != CKDA_GATES_F32);
  return extra == 0 ? core : ((core + 255) & ~size_t(255)) + extra;
}

}  // extern "C"

namespace {

constexpr int kPrepare = 1, kFinish = 2;

// Host validation shared by the chunked-forward entry points.  `passes` says
// which tensors the call uses: kPrepare needs q, k, alpha, beta; kFinish
// needs v and o (and reads h0, writes ht).  Pointers a pass does not use must
// be NULL.
ckda_status_t validate_fwd(const ckda_fwd_desc_t* d, const void* q, const void* k,
                           const void* v, const void* alpha, const void* beta,
                           const int32_t* cu_seqlens, const float* h0, const void* o,
                           const float* ht, const void* workspace, size_t workspace_bytes,
                           int passes, bool check_workspace = true) {
  if (!d) return fail(CKDA_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->B <= 0 || d->T < 0 || d->H <= 0 || d->dk <= 0 || d->dv <= 0 || d->num_seqs < 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT,
                "non-positive size: B=%d T=%d H=%d dk=%d dv=%d num_seqs=%d", d->B, d->T, d->H,
                d->dk, d->dv, d->num_seqs);
  if (d->io_dtype != CKDA_DTYPE_BF16 && d->io_dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not a ckda_dtype_t", d->io_dtype);
  if (d->gate_range != CKDA_GATE_KDA && d->gate_range != CKDA_GATE_CKDA)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "gate_range %d is not a ckda_gate_t", d->gate_range);
  if (!valid_gate_input(d->gate_input))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "gate_input %d is not a ckda_gate_input_t",
                d->gate_input);
  if (!valid_qk_heads(d->H, d->qk_heads))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "qk_heads %d does not divide H=%d", d->qk_heads, d->H);
  if (d->sign_absorb != 0 && d->sign_absorb != 1)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "sign_absorb must be 0 or 1");
  if (d->use_qk_l2norm != 0 && d->use_qk_l2norm != 1)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "use_qk_l2norm must be 0 or 1");
  if (d->chunk_size != 16 && d->chunk_size != 32 && d->chunk_size != 64)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "chunk_size %d is not 16, 32 or 64", d->chunk_size);
  if (cu_seqlens) {
    if (d->B != 1)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "cu_seqlens given with B=%d (must be 1)", d->B);
    if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "cu_seqlens is not 4-byte aligned");
  } else if (d->num_seqs != d->B) {
    return fail(CKDA_ERR_INVALID_ARGUMENT, "num_seqs=%d must equal B=%d without cu_seqlens",
                d->num_seqs, d->B);
  }
  const int64_t tokens = static_cast<int64_t>(d->B) * d->T;
  if (tokens > 0 && (passes & kPrepare) && (!q || !k || !alpha || !beta))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "q, k, alpha and beta must not be NULL");
  if (tokens > 0 && (passes & kFinish) && (!v || !o))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "v and o must not be NULL");
  const void* ptrs[] = {q, k, v, alpha, beta, h0, o, ht};
  const char* names[] = {"q", "k", "v", "alpha", "beta", "h0", "o", "ht"};
  for (int i = 0; i < 8; ++i)
    if (ptrs[i] && !aligned16(ptrs[i]))
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", names[i]);

  const int64_t eb = elem_bytes(d->io_dtype);
  const int64_t gb = gate_bytes(d->gate_input);
  const int64_t hk = qk_heads_of(d->H, d->qk_heads);
  const int64_t state_bytes = static_cast<int64_t>(d->num_seqs) * d->H * d->dk * d->dv * 4;
  const Range ro = range("o", o, o ? tokens * d->H * d->dv * eb : 0);
  const Range ins[] = {range("q", q, q ? tokens * hk * d->dk * eb : 0),
                       range("k", k, k ? tokens * hk * d->dk * eb : 0),
                       range("v", v, v ? tokens * d->H * d->dv * eb : 0),
                       range("alpha", alpha, alpha ? tokens * d->H * d->dk * gb : 0),
                       range("beta", beta, beta ? tokens * d->H * gb : 0),
                       range("h0", h0, h0 ? state_bytes : 0),
                       range("ht", ht, ht ? state_bytes : 0),
                       range("cu_seqlens", cu_seqlens,
                             cu_seqlens ? 4 * (static_cast<int64_t>(d->num_seqs) + 1) : 0)};
  for (const Range& r : ins)
    if (overlap(ro, r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "o overlaps %s", r.name);
  if (ht) {
    const Range rh = range("ht", ht, state_bytes);
    for (int i = 0; i < 5; ++i)
      if (overlap(rh, ins[i])) return fail(CKDA_ERR_INVALID_ARGUMENT, "ht overlaps %s", ins[i].name);
    if (h0 && h0 != ht && overlap(rh, ins[5]))
      return fail(CKDA_ERR_INVALID_ARGUMENT, "ht partially overlaps h0");
  }
  const size_t need = check_workspace ? ckda_chunk_fwd_workspace_size(d, cu_seqlens ? 1 : 0) : 0;
  if (need > 0) {
    if (!workspace)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace is NULL (%zu bytes needed)", need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace is not 256-byte aligned");
    if (workspace_bytes < need)
      return fail(CKDA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, %zu needed",
                  workspace_bytes, need);
    const Range rw = range("workspace", workspace, static_cast<int64_t>(need));
    if (overlap(rw, ro)) return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace overlaps o");
    for (const Range& r : ins)
      if (overlap(rw, r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace overlaps %s", r.name);
  }
  if (!ckda::fwd_supported(d->chunk_size, d->dk, d->dv, d->io_dtype))
    return fail(CKDA_ERR_UNSUPPORTED, "no chunked kernel for chunk_size=%d dk=%d dv=%d io_dtype=%d",
                d->chunk_size, d->dk, d->dv, d->io_dtype);
  return ok();
}

ckda_status_t run_fwd(const ckda_fwd_desc_t* d, const void* q, const void* k, const void* v,
                      const void* alpha, const void* beta, const int32_t* cu_seqlens,
                      const float* h0, void* o, float* ht, void* workspace, size_t workspace_bytes,
                      void* stream, int passes) {
  const ckda_status_t st = validate_fwd(d, q, k, v, alpha, beta, cu_seqlens, h0, o, ht,
                                        workspace, workspace_bytes, passes);
  if (st != CKDA_OK) return st;
  if (d->num_seqs == 0) return ok();
  ckda::FwdArgs a{d->B, d->T, d->H, d->dk, d->dv, d->num_seqs, d->chunk_size,
                  qk_heads_of(d->H, d->qk_heads), d->use_qk_l2norm, d->gate_range, d->gate_input,
                  d->sign_absorb, d->scale, q, k, v, alpha, beta,
                  cu_seqlens, h0, o, ht, nullptr, nullptr, nullptr, nullptr, 0, 0, 0};
  return from_hip(ckda::launch_fwd(a, d->io_dtype, workspace, static_cast<hipStream_t>(stream),
                                   (passes & kPrepare) != 0, (passes & kFinish) != 0));
}

// The backward takes the forward's inputs plus dout (in the place of o) and
// dht, and writes fp32 gradients.
ckda_status_t run_bwd(const ckda_fwd_desc_t* d, const void* q, const void* k, const void* v,
                      const void* alpha, const void* beta, const int32_t* cu_seqlens,
                      const float* h0, const void* dout, const float* dht, float* dq, float* dk,
                      float* dv, float* dalpha, float* dbeta, float* dh0, void* workspace,
                      size_t workspace_bytes, void* stream, bool recompute) {
  ckda_status_t st = validate_fwd(d, q, k, v, alpha, beta, cu_seqlens, h0, dout, nullptr, nullptr,
                                  0, kPrepare | kFinish, false);
  if (st != CKDA_OK) return st;
  if (d->sign_absorb != 0)
    return fail(CKDA_ERR_UNSUPPORTED, "the backward has no sign-absorption path");
  const int64_t tokens = static_cast<int64_t>(d->B) * d->T;
  if (tokens > 0 && (!dq || !dk || !dv || !dalpha || !dbeta))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "dq, dk, dv, dalpha and dbeta must not be NULL");
  const void* outp[] = {dq, dk, dv, dalpha, dbeta, dh0};
  const char* onames[] = {"dq", "dk", "dv", "dalpha", "dbeta", "dh0"};
  for (int i = 0; i < 6; ++i)
    if (outp[i] && !aligned16(outp[i]))
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", onames[i]);
  if (dht && !aligned16(dht)) return fail(CKDA_ERR_INVALID_ARGUMENT, "dht is not 16-byte aligned");
  const int64_t eb = elem_bytes(d->io_dtype), gb = gate_bytes(d->gate_input);
  const int32_t Hk = qk_heads_of(d->H, d->qk_heads);
  const int64_t state_bytes = static_cast<int64_t>(d->num_seqs) * d->H * d->dk * d->dv * 4;
  // q, k, dq, dk on the q/k heads; alpha, dalpha, beta, dbeta on the value heads
  const int64_t nqk = tokens * Hk * d->dk, na = tokens * d->H * d->dk, nv = tokens * d->H * d->dv;
  const Range outs[] = {range("dq", dq, dq ? 4 * nqk : 0), range("dk", dk, dk ? 4 * nqk : 0),
                        range("dv", dv, dv ? 4 * nv : 0), range("dalpha", dalpha, dalpha ? 4 * na : 0),
                        range("dbeta", dbeta, dbeta ? 4 * tokens * d->H : 0),
                        range("dh0", dh0, dh0 ? state_bytes : 0)};
  const Range ins[] = {range("q", q, q ? nqk * eb : 0), range("k", k, k ? nqk * eb : 0),
                       range("v", v, v ? nv * eb : 0), range("alpha", alpha, alpha ? gb * na : 0),
                       range("beta", beta, beta ? gb * tokens * d->H : 0),
                       range("h0", h0, h0 ? state_bytes : 0), range("dout", dout, dout ? nv * eb : 0),
                       range("dht", dht, dht ? state_bytes : 0),
                       range("cu_seqlens", cu_seqlens,
                             cu_seqlens ? 4 * (static_cast<int64_t>(d->num_seqs) + 1) : 0)};
  for (int i = 0; i < 6; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, r.name);
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j]))
        return fail(CKDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", outs[i].name, outs[j].name);
  }
  const size_t need = ckda_chunk_bwd_workspace_size(d, cu_seqlens ? 1 : 0);
  if (need > 0) {
    if (!workspace)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace is NULL (%zu bytes needed)", need);
    if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace is not 256-byte aligned");
    if (workspace_bytes < need)
      return fail(CKDA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, %zu needed",
                  workspace_bytes, need);
    const Range rw = range("workspace", workspace, static_cast<int64_t>(need));
    for (const Range& r : ins)
      if (overlap(rw, r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace overlaps %s", r.name);
    for (const Range& r : outs)
      if (overlap(rw, r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace overlaps %s", r.name);
  }
  if (d->num_seqs == 0) return ok();
  ckda::BwdArgs b{};
  b.f = ckda::FwdArgs{d->B, d->T, d->H, d->dk, d->dv, d->num_seqs, d->chunk_size, Hk,
                      d->use_qk_l2norm, d->gate_range, d->gate_input, 0, d->scale, q, k, v,
                      alpha, beta, cu_seqlens, h0, nullptr, nullptr};
  b.dout = dout;
  b.dht = dht;
  b.dq = dq;
  b.dk = dk;
  b.dv = dv;
  b.dalpha = dalpha;
  b.dbeta = dbeta;
  b.dh0 = dh0;
  const size_t core = ckda::bwd_workspace_bytes(d->B, d->T, d->H, d->dk, d->dv, d->num_seqs,
                                                d->chunk_size, d->io_dtype, cu_seqlens != nullptr);
  return from_hip(ckda::launch_bwd_full(b, d->io_dtype, workspace, core,
                                        static_cast<hipStream_t>(stream), recompute));
}

// The forward that also keeps the backward's records in `saved` (laid out as
// the backward's workspace), for ckda_chunk_bwd_saved.
ckda_status_t run_fwd_save(const ckda_fwd_desc_t* d, const void* q, const void* k, const void* v,
                           const void* alpha, const void* beta, const int32_t* cu_seqlens,
                           const float* h0, void* o, float* ht, void* saved, size_t saved_bytes,
                           void* stream) {
  ckda_status_t st = validate_fwd(d, q, k, v, alpha, beta, cu_seqlens, h0, o, ht, nullptr, 0,
                                  kPrepare | kFinish, false);
  if (st != CKDA_OK) return st;
  if (d->sign_absorb != 0)
    return fail(CKDA_ERR_UNSUPPORTED, "the backward's records have no sign-absorption path");
  const int64_t tokens = static_cast<int64_t>(d->B) * d->T;
  const int64_t eb = elem_bytes(d->io_dtype), gb = gate_bytes(d->gate_input);
  const int32_t Hk = qk_heads_of(d->H, d->qk_heads);
  const int64_t state_bytes = static_cast<int64_t>(d->num_seqs) * d->H * d->dk * d->dv * 4;
  const int64_t nqk = tokens * Hk * d->dk, na = tokens * d->H * d->dk, nv = tokens * d->H * d->dv;
  const Range others[] = {range("q", q, q ? nqk * eb : 0), range("k", k, k ? nqk * eb : 0),
                          range("v", v, v ? nv * eb : 0), range("alpha", alpha, alpha ? gb * na : 0),
                          range("beta", beta, beta ? gb * tokens * d->H : 0),
                          range("h0", h0, h0 ? state_bytes : 0), range("o", o, o ? nv * eb : 0),
                          range("ht", ht, ht ? state_bytes : 0),
                          range("cu_seqlens", cu_seqlens,
                                cu_seqlens ? 4 * (static_cast<int64_t>(d->num_seqs) + 1) : 0)};
  const size_t need = ckda_chunk_bwd_workspace_size(d, cu_seqlens ? 1 : 0);
  if (need > 0) {
    if (!saved) return fail(CKDA_ERR_INVALID_ARGUMENT, "saved is NULL (%zu bytes needed)", need);
    if ((reinterpret_cast<uintptr_t>(saved) & 255u) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "saved is not 256-byte aligned");
    if (saved_bytes < need)
      return fail(CKDA_ERR_WORKSPACE_TOO_SMALL, "saved has %zu bytes, %zu needed", saved_bytes, need);
    const Range rs = range("saved", saved, static_cast<int64_t>(need));
    for (const Range& r : others)
      if (overlap(rs, r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "saved overlaps %s", r.name);
  }
  if (d->num_seqs == 0) return ok();
  ckda::FwdArgs a{d->B, d->T, d->H, d->dk, d->dv, d->num_seqs, d->chunk_size, Hk,
                  d->use_qk_l2norm, d->gate_range, d->gate_input, 0, d->scale, q, k, v, alpha,
                  beta, cu_seqlens, h0, o, ht, nullptr, nullptr, nullptr, nullptr, 0, 0, 0};
  return from_hip(ckda::launch_fwd_save(a, d->io_dtype, saved, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

ckda_status_t ckda_chunk_bwd(const ckda_fwd_desc_t* d, const void* q, const void* k,
                             const void* v, const void* alpha, const void* beta,
                             const int32_t* cu_seqlens, const float* h0, const void* dout,
                             const float* dht, float* dq, float* dk, float* dv, float* dalpha,
                             float* dbeta, float* dh0, void* workspace, size_t workspace_bytes,
                             void* stream) {
  return run_bwd(d, q, k, v, alpha, beta, cu_seqlens, h0, dout, dht, dq, dk, dv, dalpha, dbeta,
                 dh0, workspace, workspace_bytes, stream, true);
}

ckda_status_t ckda_chunk_fwd_save(const ckda_fwd_desc_t* d, const void* q, const void* k,
                                  const void* v, const void* alpha, const void* beta,
                                  const int32_t* cu_seqlens, const float* h0, void* o, float* ht,
                                  void* saved, size_t saved_bytes, void* stream) {
  return run_fwd_save(d, q, k, v, alpha, beta, cu_seqlens, h0, o, ht, saved, saved_bytes, stream);
}

ckda_status_t ckda_chunk_bwd_saved(const ckda_fwd_desc_t* d, const void* q, const void* k,
                                   const void* v, const void* alpha, const void* beta,
                                   const int32_t* cu_seqlens, const float* h0, const void* dout,
                                   const float* dht, float* dq, float* dk, float* dv,
                                   float* dalpha, float* dbeta, float* dh0, void* saved,
                                   size_t saved_bytes, void* stream) {
  return run_bwd(d, q, k, v, alpha, beta, cu_seqlens, h0, dout, dht, dq, dk, dv, dalpha, dbeta,
                 dh0, saved, saved_bytes, stream, false);
}

ckda_status_t ckda_chunk_fwd(const ckda_fwd_desc_t* d, const void* q, const void* k,
                             const void* v, const void* alpha, const void* beta,
                             const int32_t* cu_seqlens, const float* h0, void* o,
                             float* ht, void* workspace, size_t workspace_bytes, void* stream) {
  return run_fwd(d, q, k, v, alpha, beta, cu_seqlens, h0, o, ht, workspace, workspace_bytes,
                 stream, kPrepare | kFinish);
}

ckda_status_t ckda_chunk_fwd_noalloc(const ckda_fwd_desc_t* d, const void* q, const void* k,
                                     const void* v, const void* alpha, const void* beta,
                                     const int32_t* cu_seqlens, const float* h0, void* o,
                                     float* ht, void* stream) {
  if (!d) return fail(CKDA_ERR_INVALID_ARGUMENT, "desc is NULL");
  // sizes first, on the host: a call whose workspace would not fit the
  // static scratch is refused before anything touches the GPU
  const size_t need = ckda_chunk_fwd_workspace_size(d, cu_seqlens ? 1 : 0);
  if (need > CKDA_NOALLOC_SCRATCH_BYTES)
    return fail(CKDA_ERR_WORKSPACE_TOO_SMALL,
                "this call needs %zu bytes of scratch; the static scratch of "
                "ckda_chunk_fwd_noalloc holds %zu (use ckda_chunk_fwd with a workspace)",
                need, static_cast<size_t>(CKDA_NOALLOC_SCRATCH_BYTES));
  const ckda_status_t st = validate_fwd(d, q, k, v, alpha, beta, cu_seqlens, h0, o, ht, nullptr,
                                        0, kPrepare | kFinish, false);
  if (st != CKDA_OK) return st;
  if (d->num_seqs == 0 || need == 0) return ok();
  void* ws = nullptr;
  const hipError_t e = scratch_address(static_cast<hipStream_t>(stream), &ws);
  if (e != hipSuccess)
    return fail(CKDA_ERR_HIP, "looking up the static scratch failed: HIP error %d: %s",
                static_cast<int>(e), hipGetErrorString(e));
  return run_fwd(d, q, k, v, alpha, beta, cu_seqlens, h0, o, ht, ws, CKDA_NOALLOC_SCRATCH_BYTES,
                 stream, kPrepare | kFinish);
}

ckda_status_t ckda_chunk_fwd_prepare(const ckda_fwd_desc_t* d, const void* q, const void* k,
                                     const void* alpha, const void* beta,
                                     const int32_t* cu_seqlens, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  return run_fwd(d, q, k, nullptr, alpha, beta, cu_seqlens, nullptr, nullptr, nullptr, workspace,
                 workspace_bytes, stream, kPrepare);
}

ckda_status_t ckda_chunk_fwd_finish(const ckda_fwd_desc_t* d, const void* v,
                                    const int32_t* cu_seqlens, const float* h0, void* o,
                                    float* ht, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  return run_fwd(d, nullptr, nullptr, v, nullptr, nullptr, cu_seqlens, h0, o, ht, workspace,
                 workspace_bytes, stream, kFinish);
}

ckda_status_t ckda_recurrent_step(int32_t N, int32_t H, int32_t qk_heads, int32_t dk,
                                  int32_t dv, int32_t io_dtype, int32_t gate_range, int32_t gate_input,
                                  int32_t use_qk_l2norm, float scale, const void* q,
                                  const void* k, const void* v, const void* alpha,
                                  const void* beta, const float* h0,
                                  float* ht, void* o, void* stream) {
  if (N < 0 || H <= 0 || dk <= 0 || dv <= 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "bad size: N=%d H=%d dk=%d dv=%d", N, H, dk, dv);
  if (io_dtype != CKDA_DTYPE_BF16 && io_dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not a ckda_dtype_t", io_dtype);
  if (gate_range != CKDA_GATE_KDA && gate_range != CKDA_GATE_CKDA)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "gate_range %d is not a ckda_gate_t", gate_range);
  if (!valid_gate_input(gate_input))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "gate_input %d is not a ckda_gate_input_t", gate_input);
  if (!valid_qk_heads(H, qk_heads))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "qk_heads %d does not divide H=%d", qk_heads, H);
  if (use_qk_l2norm != 0 && use_qk_l2norm != 1)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "use_qk_l2norm must be 0 or 1");
  if (N > 0 && (!q || !k || !v || !alpha || !beta || !h0 || !ht || !o))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "no pointer argument may be NULL");
  const void* ptrs[] = {q, k, v, alpha, beta, h0, ht, o};
  const char* names[] = {"q", "k", "v", "alpha", "beta", "h0", "ht", "o"};
  for (int i = 0; i < 8; ++i)
    if (ptrs[i] && !aligned16(ptrs[i]))
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", names[i]);
  const int64_t nh = static_cast<int64_t>(N) * H;
  if (nh > (int64_t(1) << 21))  // one launch of up to 2048 work-items per (sequence, head)
    return fail(CKDA_ERR_UNSUPPORTED, "N*H = %lld exceeds 2^21 for one decode launch",
                static_cast<long long>(nh));
  const int64_t nhk = static_cast<int64_t>(N) * qk_heads_of(H, qk_heads);
  const int64_t eb = elem_bytes(io_dtype);
  const int64_t gb = gate_bytes(gate_input);
  const int64_t sb = nh * dk * dv * 4;
  const Range ro = range("o", o, nh * dv * eb);
  const Range rht = range("ht", ht, sb);
  const Range ins[] = {range("q", q, nhk * dk * eb), range("k", k, nhk * dk * eb),
                       range("v", v, nh * dv * eb), range("alpha", alpha, nh * dk * gb),
                       range("beta", beta, nh * gb), range("h0", h0, sb)};
  for (const Range& r : ins)
    if (overlap(ro, r)) return fail(CKDA_ERR_INVALID_ARGUMENT, "o overlaps %s", r.name);
  if (overlap(ro, rht)) return fail(CKDA_ERR_INVALID_ARGUMENT, "o overlaps ht");
  for (int i = 0; i < 5; ++i)
    if (overlap(rht, ins[i])) return fail(CKDA_ERR_INVALID_ARGUMENT, "ht overlaps %s", ins[i].name);
  if (h0 != ht && overlap(rht, ins[5]))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "ht partially overlaps h0");
  if (!ckda::step_supported(dk, dv))
    return fail(CKDA_ERR_UNSUPPORTED, "no decode kernel for dk=%d dv=%d", dk, dv);
  if (nh == 0) return ok();
  ckda::StepArgs a{N, H, dk, dv, qk_heads_of(H, qk_heads), use_qk_l2norm, gate_range, gate_input, scale, q, k, v,
                   alpha, beta, h0, ht, o};
  return from_hip(ckda::launch_step(a, io_dtype, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_l2norm_debug(const void* x, float* y, int64_t rows, int32_t d,
                                int32_t dtype, void* stream) {
  if (rows < 0 || d <= 0 || d > 1024)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "bad size: rows=%lld d=%d",
                static_cast<long long>(rows), d);
  if (dtype != CKDA_DTYPE_BF16 && dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "dtype %d is not a ckda_dtype_t", dtype);
  if (rows > 0 && (!x || !y)) return fail(CKDA_ERR_INVALID_ARGUMENT, "x and y must not be NULL");
  if ((x && !aligned16(x)) || (y && !aligned16(y)))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "x and y must be 16-byte aligned");
  if (overlap(range("x", x, rows * d * elem_bytes(dtype)), range("y", y, rows * d * 4)))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "y overlaps x");
  if (rows == 0) return ok();
  return from_hip(ckda::launch_l2norm_debug(x, y, rows, d, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- decay linear attention ------------------------------------------------
namespace {

// The tensors of one decay call, for the checks of alignment and overlap.
struct Tensor {
  Range r;
  bool out;      // written
  bool needed;   // may not be NULL
  uint32_t align = 16;
};

// Every tensor aligned and given where needed; no output overlaps an input or
// another output, but for the pair (same_a, same_b), which may be one buffer.
ckda_status_t check_tensors(const Tensor* ts, int n, int same_a = -1, int same_b = -1) {
  for (int i = 0; i < n; ++i) {
    if (ts[i].needed && ts[i].r.lo == 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s must not be NULL", ts[i].r.name);
    if ((ts[i].r.lo & (ts[i].align - 1)) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s is not %u-byte aligned", ts[i].r.name, ts[i].align);
  }
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (!ts[i].out || i == j || (ts[j].out && j < i)) continue;
      if (ts[i].r.lo == 0 || ts[j].r.lo == 0 || !overlap(ts[i].r, ts[j].r)) continue;
      if (((i == same_a && j == same_b) || (i == same_b && j == same_a)) && ts[i].r.lo == ts[j].r.lo)
        continue;
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s overlaps %s", ts[i].r.name, ts[j].r.name);
    }
  return ok();
}

ckda_status_t check_workspace(const Tensor* ts, int n, const void* ws, size_t bytes, size_t need) {
  if (need == 0) return ok();
  if (!ws) return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace is NULL (%zu bytes needed)", need);
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace is not 256-byte aligned");
  if (bytes < need)
    return fail(CKDA_ERR_WORKSPACE_TOO_SMALL, "workspace has %zu bytes, %zu needed", bytes, need);
  const Range rw = range("workspace", ws, static_cast<int64_t>(need));
  for (int i = 0; i < n; ++i)
    if (ts[i].r.lo != 0 && overlap(rw, ts[i].r))
      return fail(CKDA_ERR_INVALID_ARGUMENT, "workspace overlaps %s", ts[i].r.name);
  return ok();
}

bool valid_decay_sizes(const ckda_decay_desc_t* d) {
  return d->B > 0 && d->T >= 0 && d->H > 0 && d->dk > 0 && d->dv > 0 && d->num_seqs >= 0 &&
         (d->io_dtype == CKDA_DTYPE_BF16 || d->io_dtype == CKDA_DTYPE_F32) &&
         valid_qk_heads(d->H, d->qk_heads) && valid_gate_input(d->gate_input);
}

ckda::DecayArgs decay_args(const ckda_decay_desc_t* d, const int32_t* cu) {
  ckda::DecayArgs a{};
  a.B = d->B;
  a.T = d->T;
  a.H = d->H;
  a.Hk = qk_heads_of(d->H, d->qk_heads);
  a.dk = d->dk;
  a.dv = d->dv;
  a.N = d->num_seqs;
  a.gate_range = d->gate_range;
  a.gate_input = d->gate_input;
  a.per_head = d->alpha_per_head;
  a.scale = d->scale;
  a.cu = cu;
  return a;
}

ckda_status_t validate_decay(const ckda_decay_desc_t* d, const int32_t* cu, ckda::DecayCall call) {
  if (!d) return fail(CKDA_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->B <= 0 || d->T < 0 || d->H <= 0 || d->dk <= 0 || d->dv <= 0 || d->num_seqs < 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT,
                "non-positive size: B=%d T=%d H=%d dk=%d dv=%d num_seqs=%d", d->B, d->T, d->H,
                d->dk, d->dv, d->num_seqs);
  if (d->io_dtype != CKDA_DTYPE_BF16 && d->io_dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not a ckda_dtype_t", d->io_dtype);
  if (d->gate_range != CKDA_GATE_KDA && d->gate_range != CKDA_GATE_CKDA)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "gate_range %d is not a ckda_gate_t", d->gate_range);
  if (!valid_gate_input(d->gate_input))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "gate_input %d is not a ckda_gate_input_t", d->gate_input);
  if (d->alpha_per_head != 0 && d->alpha_per_head != 1)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "alpha_per_head must be 0 or 1");
  if (!valid_qk_heads(d->H, d->qk_heads))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "qk_heads %d does not divide H=%d", d->qk_heads, d->H);
  if (cu) {
    if (d->B != 1)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "cu_seqlens given with B=%d (must be 1)", d->B);
    if ((reinterpret_cast<uintptr_t>(cu) & 3u) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "cu_seqlens is not 4-byte aligned");
  } else if (d->num_seqs != d->B) {
    return fail(CKDA_ERR_INVALID_ARGUMENT, "num_seqs=%d must equal B=%d without cu_seqlens",
                d->num_seqs, d->B);
  }
  if (!ckda::decay_supported(d->dk, d->dv))
    return fail(CKDA_ERR_UNSUPPORTED, "no decay kernel for dk=%d dv=%d (multiples of 8 up to 128)",
                d->dk, d->dv);
  // a chunk's rows of one tensor are addressed with 32-bit offsets
  if (static_cast<int64_t>(d->H) * (d->dk > d->dv ? d->dk : d->dv) >= (int64_t(1) << 22))
    return fail(CKDA_ERR_UNSUPPORTED, "H * max(dk, dv) of 2^22 or more");
  // walks look two chunks past the end
  if (static_cast<int64_t>(d->B) * d->T >= (int64_t(1) << 31) - 1024 ||
      ckda::decay_grid(decay_args(d, cu), d->io_dtype) >= (int64_t(1) << 31) ||
      ckda::decay_threads(decay_args(d, cu), d->io_dtype, call) >= (int64_t(1) << 32))
    return fail(CKDA_ERR_UNSUPPORTED, "too many (sequence, head) chunks for one launch");
  return ok();
}

struct DecaySizes {
  int64_t tokens, qk, vo, alpha, state;  // elements, elements, elements, bytes, bytes
  int64_t es;
};
DecaySizes decay_sizes(const ckda_decay_desc_t* d) {
  DecaySizes z;
  z.tokens = static_cast<int64_t>(d->B) * d->T;
  z.es = elem_bytes(d->io_dtype);
  z.qk = z.tokens * qk_heads_of(d->H, d->qk_heads) * d->dk;
  z.vo = z.tokens * d->H * d->dv;
  z.alpha = (d->alpha_per_head ? 1 : z.tokens) * d->H * gate_bytes(d->gate_input);
  z.state = static_cast<int64_t>(d->num_seqs) * d->H * d->dk * d->dv * 4;
  return z;
}

}  // namespace

extern "C" {

int32_t ckda_decay_supported(int32_t dk, int32_t dv) { return ckda::decay_supported(dk, dv) ? 1 : 0; }

size_t ckda_decay_fwd_workspace_size(const ckda_decay_desc_t* d, int32_t packed) {
  if (!d || !valid_decay_sizes(d) || !ckda::decay_supported(d->dk, d->dv) || d->num_seqs == 0) return 0;
  static const int32_t given = 0;  // only whether the batch is packed matters here
  return ckda::decay_segment_bytes(decay_args(d, packed ? &given : nullptr));
}

size_t ckda_decay_bwd_workspace_size(const ckda_decay_desc_t* d, int32_t packed) {
  if (!d || !valid_decay_sizes(d) || !ckda::decay_supported(d->dk, d->dv) || d->num_seqs == 0) return 0;
  static const int32_t given = 0;
  return ckda::decay_bwd_workspace(decay_args(d, packed ? &given : nullptr), d->io_dtype);
}

ckda_status_t ckda_decay_fwd(const ckda_decay_desc_t* d, const void* q, const void* k, const void* v,
                             const void* alpha, const int32_t* cu_seqlens, const float* h0, void* o,
                             float* ht, void* workspace, size_t workspace_bytes, void* stream) {
  ckda_status_t st = validate_decay(d, cu_seqlens, ckda::kDecayFwd);
  if (st != CKDA_OK) return st;
  const DecaySizes z = decay_sizes(d);
  const bool some = z.tokens > 0;
  const Tensor ts[] = {{range("q", q, q ? z.qk * z.es : 0), false, some},
                       {range("k", k, k ? z.qk * z.es : 0), false, some},
                       {range("v", v, v ? z.vo * z.es : 0), false, some},
                       {range("alpha", alpha, alpha ? z.alpha : 0), false, some},
                       {range("h0", h0, h0 ? z.state : 0), false, false},
                       {range("o", o, o ? z.vo * z.es : 0), true, some},
                       {range("ht", ht, ht ? z.state : 0), true, false}};
  if ((st = check_tensors(ts, 7, 4, 6)) != CKDA_OK) return st;
  if (cu_seqlens) {
    const Range rc = range("cu_seqlens", cu_seqlens, 4 * (static_cast<int64_t>(d->num_seqs) + 1));
    for (int i = 5; i < 7; ++i)
      if (overlap(ts[i].r, rc))
        return fail(CKDA_ERR_INVALID_ARGUMENT, "%s overlaps cu_seqlens", ts[i].r.name);
  }
  const size_t need = ckda_decay_fwd_workspace_size(d, cu_seqlens ? 1 : 0);
  if ((st = check_workspace(ts, 7, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  if (d->num_seqs == 0) return ok();
  ckda::DecayArgs a = decay_args(d, cu_seqlens);
  a.q = q;
  a.k = k;
  a.v = v;
  a.alpha = alpha;
  a.h0 = h0;
  a.o = o;
  a.ht = ht;
  return from_hip(ckda::launch_decay_fwd(a, d->io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_decay_bwd(const ckda_decay_desc_t* d, const void* q, const void* k, const void* v,
                             const void* alpha, const int32_t* cu_seqlens, const float* h0,
                             const void* dout, const float* dht, void* dq, void* dk, void* dv,
                             void* dalpha, float* dh0, void* workspace, size_t workspace_bytes,
                             void* stream) {
  ckda_status_t st = validate_decay(d, cu_seqlens, ckda::kDecayBwd);
  if (st != CKDA_OK) return st;
  const DecaySizes z = decay_sizes(d);
  const bool some = z.tokens > 0;
  const int64_t da = (d->alpha_per_head ? 1 : z.tokens) * d->H * z.es;
  const Tensor ts[] = {{range("q", q, q ? z.qk * z.es : 0), false, some},
                       {range("k", k, k ? z.qk * z.es : 0), false, some},
                       {range("v", v, v ? z.vo * z.es : 0), false, some},
                       {range("alpha", alpha, alpha ? z.alpha : 0), false, some},
                       {range("h0", h0, h0 ? z.state : 0), false, false},
                       {range("dout", dout, dout ? z.vo * z.es : 0), false, some},
                       {range("dht", dht, dht ? z.state : 0), false, false},
                       {range("dq", dq, dq ? z.qk * z.es : 0), true, some},
                       {range("dk", dk, dk ? z.qk * z.es : 0), true, some},
                       {range("dv", dv, dv ? z.vo * z.es : 0), true, some},
                       {range("dalpha", dalpha, dalpha ? da : 0), true, false},
                       {range("dh0", dh0, dh0 ? z.state : 0), true, false}};
  if ((st = check_tensors(ts, 12)) != CKDA_OK) return st;
  if (cu_seqlens) {
    const Range rc = range("cu_seqlens", cu_seqlens, 4 * (static_cast<int64_t>(d->num_seqs) + 1));
    for (int i = 7; i < 12; ++i)
      if (overlap(ts[i].r, rc))
        return fail(CKDA_ERR_INVALID_ARGUMENT, "%s overlaps cu_seqlens", ts[i].r.name);
  }
  const size_t need = ckda_decay_bwd_workspace_size(d, cu_seqlens ? 1 : 0);
  if ((st = check_workspace(ts, 12, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  ckda::DecayArgs a = decay_args(d, cu_seqlens);
  a.q = q;
  a.k = k;
  a.v = v;
  a.alpha = alpha;
  a.h0 = h0;
  ckda::DecayGrads g{dout, dht, dq, dk, dv, dalpha, dh0, nullptr};
  return from_hip(ckda::launch_decay_bwd(a, g, d->io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_decay_step(int32_t N, int32_t H, int32_t qk_heads, int32_t dk, int32_t dv,
                              int32_t io_dtype, int32_t gate_range, int32_t gate_input,
                              int32_t alpha_per_head, float scale, const void* q, const void* k,
                              const void* v, const void* alpha, const float* h0, float* ht, void* o,
                              void* stream) {
  if (N < 0 || H <= 0 || dk <= 0 || dv <= 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "bad size: N=%d H=%d dk=%d dv=%d", N, H, dk, dv);
  // one token a sequence is a dense batch of N sequences of one token
  const ckda_decay_desc_t d{N > 0 ? N : 1, 1, H, dk, dv, N > 0 ? N : 1, io_dtype, gate_range,
                            gate_input, qk_heads, alpha_per_head, scale};
  ckda_status_t st = validate_decay(&d, nullptr, ckda::kDecayStep);
  if (st != CKDA_OK) return st;
  const int64_t nh = static_cast<int64_t>(N) * H;
  if (nh > (int64_t(1) << 21))
    return fail(CKDA_ERR_UNSUPPORTED, "N*H = %lld exceeds 2^21 for one decode launch",
                static_cast<long long>(nh));
  const DecaySizes z = decay_sizes(&d);
  const bool some = N > 0;
  const Tensor ts[] = {{range("q", q, z.qk * z.es), false, some},
                       {range("k", k, z.qk * z.es), false, some},
                       {range("v", v, z.vo * z.es), false, some},
                       {range("alpha", alpha, z.alpha), false, some},
                       {range("h0", h0, z.state), false, some},
                       {range("o", o, z.vo * z.es), true, some},
                       {range("ht", ht, z.state), true, some}};
  if ((st = check_tensors(ts, 7, 4, 6)) != CKDA_OK) return st;
  if (N == 0) return ok();
  ckda::DecayArgs a = decay_args(&d, nullptr);
  a.q = q;
  a.k = k;
  a.v = v;
  a.alpha = alpha;
  a.h0 = h0;
  a.o = o;
  a.ht = ht;
  return from_hip(ckda::launch_decay_step(a, io_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- norms around a block -----------------------------------------------------
namespace {

ckda_status_t validate_norm(int64_t rows, int32_t d, int32_t io_dtype, int32_t act, float eps,
                            const void* g) {
  if (rows < 0 || d <= 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "bad size: rows=%lld d=%d", static_cast<long long>(rows), d);
  if (io_dtype != CKDA_DTYPE_BF16 && io_dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not a ckda_dtype_t", io_dtype);
  if (act < CKDA_NORM_GATE_NONE || act > CKDA_NORM_GATE_SILU)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "act %d is not a ckda_norm_act_t", act);
  if (rows > 0 && (act == CKDA_NORM_GATE_NONE) != (g == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "g is given exactly with an activation");
  if (!(eps >= 0.f) || eps > 3.0e38f)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "eps must be finite and not negative");
  if (d > 16384) return fail(CKDA_ERR_UNSUPPORTED, "no norm kernel for d=%d (at most 16384)", d);
  if (rows > (int64_t(1) << 46) / d)
    return fail(CKDA_ERR_UNSUPPORTED, "rows * d is over 2^46");
  return ok();
}

}  // namespace

extern "C" {

size_t ckda_block_norm_bwd_workspace_size(int64_t rows, int32_t d, int32_t io_dtype) {
  if (rows <= 0 || d <= 0 || d > 16384) return 0;
  if (io_dtype != CKDA_DTYPE_BF16 && io_dtype != CKDA_DTYPE_F32) return 0;
  return ckda::norm_bwd_workspace(rows, d, io_dtype);
}

ckda_status_t ckda_block_norm(int64_t rows, int32_t d, int32_t io_dtype, int32_t act, float eps,
                              const void* y, const float* w, const void* g, const void* x,
                              const float* s, const float* w2, void* h, void* n, void* stream) {
  ckda_status_t st = validate_norm(rows, d, io_dtype, act, eps, g);
  if (st != CKDA_OK) return st;
  if ((w2 == nullptr) != (n == nullptr) && rows > 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "n is given exactly with w2");
  const int64_t b = rows * d * elem_bytes(io_dtype), v = 4 * static_cast<int64_t>(d);
  const bool some = rows > 0;
  const Tensor ts[] = {{range("y", y, y ? b : 0), false, some}, {range("w", w, w ? v : 0), false, false},
                       {range("g", g, g ? b : 0), false, false}, {range("x", x, x ? b : 0), false, false},
                       {range("s", s, s ? v : 0), false, false}, {range("w2", w2, w2 ? v : 0), false, false},
                       {range("h", h, h ? b : 0), true, some},   {range("n", n, n ? b : 0), true, false}};
  if ((st = check_tensors(ts, 8, 3, 6)) != CKDA_OK) return st;
  if (rows == 0) return ok();
  const ckda::NormArgs a{rows, d, act, eps, y, w, g, x, s, w2, h, n};
  return from_hip(ckda::launch_norm_fwd(a, io_dtype, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_block_norm_bwd(int64_t rows, int32_t d, int32_t io_dtype, int32_t act, float eps,
                                  const void* y, const float* w, const void* g, const void* x,
                                  const float* s, const float* w2, const void* dh, const void* dn,
                                  void* dy, float* dw, void* dg, void* dx, float* ds, float* dw2,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  ckda_status_t st = validate_norm(rows, d, io_dtype, act, eps, g);
  if (st != CKDA_OK) return st;
  if (rows == 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "no rows: the sums over rows would not be written");
  if ((w2 == nullptr) != (dn == nullptr) || (w2 == nullptr) != (dw2 == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "dn and dw2 are given exactly with w2");
  if ((w == nullptr) != (dw == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "dw is given exactly with w");
  if ((s == nullptr) != (ds == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "ds is given exactly with s");
  if ((g == nullptr) != (dg == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "dg is given exactly with g");
  const int64_t b = rows * d * elem_bytes(io_dtype), v = 4 * static_cast<int64_t>(d);
  const Tensor ts[] = {{range("y", y, y ? b : 0), false, true},   {range("w", w, w ? v : 0), false, false},
                       {range("g", g, g ? b : 0), false, false},  {range("x", x, x ? b : 0), false, false},
                       {range("s", s, s ? v : 0), false, false},  {range("w2", w2, w2 ? v : 0), false, false},
                       {range("dh", dh, dh ? b : 0), false, true}, {range("dn", dn, dn ? b : 0), false, false},
                       {range("dy", dy, dy ? b : 0), true, true}, {range("dw", dw, dw ? v : 0), true, false},
                       {range("dg", dg, dg ? b : 0), true, false}, {range("dx", dx, dx ? b : 0), true, false},
                       {range("ds", ds, ds ? v : 0), true, false}, {range("dw2", dw2, dw2 ? v : 0), true, false}};
  if ((st = check_tensors(ts, 14)) != CKDA_OK) return st;
  const size_t need = ckda_block_norm_bwd_workspace_size(rows, d, io_dtype);
  if ((st = check_workspace(ts, 14, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const ckda::NormArgs a{rows, d, act, eps, y, w, g, x, s, w2, nullptr, nullptr};
  const ckda::NormGrads gr{dh, dn, dy, dw, dg, dx, ds, dw2, nullptr};
  return from_hip(ckda::launch_norm_bwd(a, gr, io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- short convolution ----------------------------------------------------------
namespace {

// What the calls on sequences of tokens share: the batch, its packing and its size.
ckda_status_t validate_batch(int32_t B, int32_t T, int32_t num_seqs, int32_t io_dtype, const int32_t* cu) {
  if (io_dtype != CKDA_DTYPE_BF16 && io_dtype != CKDA_DTYPE_F32)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "io_dtype %d is not a ckda_dtype_t", io_dtype);
  if (cu) {
    if (B != 1) return fail(CKDA_ERR_INVALID_ARGUMENT, "cu_seqlens given with B=%d (must be 1)", B);
    if ((reinterpret_cast<uintptr_t>(cu) & 3u) != 0)
      return fail(CKDA_ERR_INVALID_ARGUMENT, "cu_seqlens is not 4-byte aligned");
  } else if (num_seqs != B) {
    return fail(CKDA_ERR_INVALID_ARGUMENT, "num_seqs=%d must equal B=%d without cu_seqlens", num_seqs, B);
  }
  // walks look ahead, and a sequence and its longest piece are added in 32 bits
  if (static_cast<int64_t>(B) * T >= (int64_t(1) << 31) - 1024 || T >= (1 << 30) ||
      static_cast<int64_t>(num_seqs) + T >= (int64_t(1) << 31))
    return fail(CKDA_ERR_UNSUPPORTED, "too many tokens for one launch");
  return ok();
}

// The elements between tokens of rows of `width`, 0 meaning contiguous rows.
bool stride_of(int64_t given, int64_t width, int64_t* stride) {
  *stride = given == 0 ? width : given;
  return *stride >= width;
}
constexpr int64_t kMaxStride = int64_t(1) << 24;  // a tile of 32 rows is addressed in 31 bits

// A tensor of `tokens` rows of `width` elements, `stride` apart.
Range rows_range(const char* name, const void* p, int64_t tokens, int64_t stride, int64_t width, int64_t es) {
  return range(name, p, p && tokens > 0 ? ((tokens - 1) * stride + width) * es : 0);
}

ckda_status_t no_output_on(const Tensor* ts, int n, const int32_t* cu, int32_t num_seqs) {
  if (!cu) return ok();
  const Range rc = range("cu_seqlens", cu, 4 * (static_cast<int64_t>(num_seqs) + 1));
  for (int i = 0; i < n; ++i)
    if (ts[i].out && overlap(ts[i].r, rc))
      return fail(CKDA_ERR_INVALID_ARGUMENT, "%s overlaps cu_seqlens", ts[i].r.name);
  return ok();
}

ckda_status_t validate_conv(const ckda_conv_desc_t* d, const int32_t* cu, bool grads, ckda::ConvArgs* a) {
  if (!d) return fail(CKDA_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->B <= 0 || d->T < 0 || d->D <= 0 || d->K <= 0 || d->num_seqs < 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "non-positive size: B=%d T=%d D=%d K=%d num_seqs=%d", d->B, d->T, d->D,
                d->K, d->num_seqs);
  if (d->act != CKDA_NORM_GATE_NONE && d->act != CKDA_NORM_GATE_SILU)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "act %d is neither none nor silu", d->act);
  const ckda_status_t st = validate_batch(d->B, d->T, d->num_seqs, d->io_dtype, cu);
  if (st != CKDA_OK) return st;
  *a = ckda::ConvArgs{};
  if (!stride_of(d->x_stride, d->D, &a->sx))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "x_stride is below D=%d", d->D);
  if (d->K < 2 || d->K > 4) return fail(CKDA_ERR_UNSUPPORTED, "no convolution kernel for K=%d (2 to 4)", d->K);
  if (d->D > (1 << 22) || a->sx >= kMaxStride)
    return fail(CKDA_ERR_UNSUPPORTED, "D over 2^22 or x_stride of 2^24 or more");
  a->B = d->B;
  a->T = d->T;
  a->D = d->D;
  a->K = d->K;
  a->N = d->num_seqs;
  a->act = d->act == CKDA_NORM_GATE_SILU;
  a->cu = cu;
  if (ckda::conv_threads(*a, grads) >= (int64_t(1) << 32))
    return fail(CKDA_ERR_UNSUPPORTED, "too many tokens and channels for one launch");
  return ok();
}

}  // namespace

extern "C" {

size_t ckda_conv_bwd_workspace_size(const ckda_conv_desc_t* d, int32_t packed) {
  static const int32_t given = 0;  // only whether the batch is packed matters here
  ckda::ConvArgs a;
  std::string kept;  // a size that is asked for is no failed call
  kept.swap(g_last_error);
  const ckda_status_t st = validate_conv(d, packed ? &given : nullptr, true, &a);
  kept.swap(g_last_error);
  return st == CKDA_OK ? ckda::conv_bwd_workspace(a) : 0;
}

ckda_status_t ckda_conv_fwd(const ckda_conv_desc_t* d, const void* x, const float* w, const float* bias,
                            const int32_t* cu_seqlens, const void* h0, void* y, void* ht, void* stream) {
  ckda::ConvArgs a;
  ckda_status_t st = validate_conv(d, cu_seqlens, false, &a);
  if (st != CKDA_OK) return st;
  const int64_t es = elem_bytes(d->io_dtype), tokens = static_cast<int64_t>(d->B) * d->T;
  const int64_t state = static_cast<int64_t>(d->num_seqs) * (d->K - 1) * d->D * es;
  const bool some = tokens > 0;
  const Tensor ts[] = {{rows_range("x", x, tokens, a.sx, d->D, es), false, some, static_cast<uint32_t>(es)},
                       {range("w", w, w ? 4 * static_cast<int64_t>(d->D) * d->K : 0), false, true},
                       {range("bias", bias, bias ? 4 * static_cast<int64_t>(d->D) : 0), false, false},
                       {range("h0", h0, h0 ? state : 0), false, false},
                       {rows_range("y", y, tokens, d->D, d->D, es), true, some},
                       {range("ht", ht, ht ? state : 0), true, false}};
  if ((st = check_tensors(ts, 6, 3, 5)) != CKDA_OK) return st;
  if ((st = no_output_on(ts, 6, cu_seqlens, d->num_seqs)) != CKDA_OK) return st;
  if (d->num_seqs == 0) return ok();
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.h0 = h0;
  a.y = y;
  a.ht = ht;
  return from_hip(ckda::launch_conv_fwd(a, d->io_dtype, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_conv_bwd(const ckda_conv_desc_t* d, const void* x, const float* w, const float* bias,
                            const int32_t* cu_seqlens, const void* h0, const void* dy, const void* dht, void* dx,
                            float* dw, float* dbias, void* dh0, void* workspace, size_t workspace_bytes,
                            void* stream) {
  ckda::ConvArgs a;
  ckda_status_t st = validate_conv(d, cu_seqlens, true, &a);
  if (st != CKDA_OK) return st;
  const int64_t es = elem_bytes(d->io_dtype), tokens = static_cast<int64_t>(d->B) * d->T;
  const int64_t state = static_cast<int64_t>(d->num_seqs) * (d->K - 1) * d->D * es;
  const int64_t taps = 4 * static_cast<int64_t>(d->D) * d->K, vec = 4 * static_cast<int64_t>(d->D);
  const bool some = tokens > 0;
  const Tensor ts[] = {{rows_range("x", x, tokens, a.sx, d->D, es), false, some, static_cast<uint32_t>(es)},
                       {range("w", w, w ? taps : 0), false, true},
                       {range("bias", bias, bias ? vec : 0), false, false},
                       {range("h0", h0, h0 ? state : 0), false, false},
                       {rows_range("dy", dy, tokens, d->D, d->D, es), false, some},
                       {range("dht", dht, dht ? state : 0), false, false},
                       {rows_range("dx", dx, tokens, d->D, d->D, es), true, some},
                       {range("dw", dw, dw ? taps : 0), true, true},
                       {range("dbias", dbias, dbias ? vec : 0), true, false},
                       {range("dh0", dh0, dh0 ? state : 0), true, false}};
  if ((st = check_tensors(ts, 10)) != CKDA_OK) return st;
  if ((st = no_output_on(ts, 10, cu_seqlens, d->num_seqs)) != CKDA_OK) return st;
  const size_t need = ckda::conv_bwd_workspace(a);
  if ((st = check_workspace(ts, 10, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.h0 = h0;
  const ckda::ConvGrads g{dy, dht, dx, dw, dbias, dh0, nullptr};
  return from_hip(ckda::launch_conv_bwd(a, g, d->io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_conv_step(const ckda_conv_desc_t* d, const void* x, const float* w, const float* bias,
                             const void* h0, void* ht, void* y, void* stream) {
  if (d && d->B == 0 && d->num_seqs == 0) return ok();
  ckda::ConvArgs a;
  ckda_status_t st = validate_conv(d, nullptr, false, &a);
  if (st != CKDA_OK) return st;
  if (d->T != 1) return fail(CKDA_ERR_INVALID_ARGUMENT, "T=%d must be 1", d->T);
  const int64_t es = elem_bytes(d->io_dtype), state = static_cast<int64_t>(d->B) * (d->K - 1) * d->D * es;
  const Tensor ts[] = {{rows_range("x", x, d->B, a.sx, d->D, es), false, true, static_cast<uint32_t>(es)},
                       {range("w", w, 4 * static_cast<int64_t>(d->D) * d->K), false, true},
                       {range("bias", bias, bias ? 4 * static_cast<int64_t>(d->D) : 0), false, false},
                       {range("h0", h0, state), false, true},
                       {range("ht", ht, state), true, true},
                       {rows_range("y", y, d->B, d->D, d->D, es), true, true}};
  if ((st = check_tensors(ts, 6, 3, 4)) != CKDA_OK) return st;
  a.x = x;
  a.w = w;
  a.bias = bias;
  a.h0 = h0;
  a.y = y;
  a.ht = ht;
  return from_hip(ckda::launch_conv_step(a, d->io_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- selective scan ---------------------------------------------------------------
namespace {

enum ScanCall { kScanFwd, kScanBwd, kScanStep };

ckda_status_t validate_scan(const ckda_scan_desc_t* d, const int32_t* cu, ScanCall call, ckda::ScanArgs* a) {
  if (!d) return fail(CKDA_ERR_INVALID_ARGUMENT, "desc is NULL");
  if (d->B <= 0 || d->T < 0 || d->D <= 0 || d->S <= 0 || d->num_seqs < 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "non-positive size: B=%d T=%d D=%d S=%d num_seqs=%d", d->B, d->T, d->D,
                d->S, d->num_seqs);
  if (d->groups <= 0 || d->D % d->groups != 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "groups %d does not divide D=%d", d->groups, d->D);
  if (d->softplus != 0 && d->softplus != 1) return fail(CKDA_ERR_INVALID_ARGUMENT, "softplus must be 0 or 1");
  const ckda_status_t st = validate_batch(d->B, d->T, d->num_seqs, d->io_dtype, cu);
  if (st != CKDA_OK) return st;
  if (!ckda::scan_supported(d->S)) return fail(CKDA_ERR_UNSUPPORTED, "no scan kernel for S=%d (1 to 64)", d->S);
  if (d->D > (1 << 20)) return fail(CKDA_ERR_UNSUPPORTED, "D over 2^20");
  *a = ckda::ScanArgs{};
  const int64_t bc = static_cast<int64_t>(d->groups) * d->S;
  if (!stride_of(d->x_stride, d->D, &a->sx) || !stride_of(d->dt_stride, d->D, &a->sdt) ||
      !stride_of(d->z_stride, d->D, &a->sz) || !stride_of(d->b_stride, bc, &a->sb) ||
      !stride_of(d->c_stride, bc, &a->sc))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "a stride is below its row");
  for (int64_t s : {a->sx, a->sdt, a->sz, a->sb, a->sc})
    if (s >= kMaxStride) return fail(CKDA_ERR_UNSUPPORTED, "a stride of 2^24 or more");
  a->B = d->B;
  a->T = d->T;
  a->D = d->D;
  a->S = d->S;
  a->G = d->groups;
  a->N = d->num_seqs;
  a->softplus = d->softplus;
  a->cu = cu;
  if ((call == kScanStep ? ckda::scan_step_threads(*a) : ckda::scan_threads(*a)) >= (int64_t(1) << 32))
    return fail(CKDA_ERR_UNSUPPORTED, "too many tokens and channels for one launch");
  return ok();
}

size_t scan_workspace(const ckda_scan_desc_t* d, int32_t packed, ScanCall call) {
  static const int32_t given = 0;  // only whether the batch is packed matters here
  ckda::ScanArgs a;
  std::string kept;  // a size that is asked for is no failed call
  kept.swap(g_last_error);
  const ckda_status_t st = validate_scan(d, packed ? &given : nullptr, call, &a);
  kept.swap(g_last_error);
  if (st != CKDA_OK || (call == kScanFwd && d->num_seqs == 0)) return 0;
  return call == kScanFwd ? ckda::scan_fwd_workspace(a) : ckda::scan_bwd_workspace(a);
}

struct ScanSizes {
  int64_t es, tokens, bc, state, A, vec;  // bytes of an element, tokens, states of a token's groups; bytes
};
ScanSizes scan_sizes(const ckda_scan_desc_t* d) {
  ScanSizes z;
  z.es = elem_bytes(d->io_dtype);
  z.tokens = static_cast<int64_t>(d->B) * d->T;
  z.bc = static_cast<int64_t>(d->groups) * d->S;
  z.A = 4 * static_cast<int64_t>(d->D) * d->S;
  z.state = z.A * d->num_seqs;
  z.vec = 4 * static_cast<int64_t>(d->D);
  return z;
}

// Whether a thread's channels can move at once: every base and stride a multiple of
// their size, and every group's channels whole vectors.
bool scan_vec(const ckda::ScanArgs& a, int64_t es) {
  const int64_t n = 4;  // a thread's channels at most, in either type
  const auto fits = [&](const void* p, int64_t stride) {
    return reinterpret_cast<uintptr_t>(p) % (n * es) == 0 && stride % n == 0;
  };
  return (a.D / a.G) % n == 0 && fits(a.x, a.sx) && fits(a.dt, a.sdt) && (!a.z || fits(a.z, a.sz));
}

}  // namespace

extern "C" {

int32_t ckda_scan_supported(int32_t S) { return ckda::scan_supported(S) ? 1 : 0; }

size_t ckda_scan_fwd_workspace_size(const ckda_scan_desc_t* d, int32_t packed) {
  return scan_workspace(d, packed, kScanFwd);
}
size_t ckda_scan_bwd_workspace_size(const ckda_scan_desc_t* d, int32_t packed) {
  return scan_workspace(d, packed, kScanBwd);
}

ckda_status_t ckda_scan_fwd(const ckda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                            const int32_t* cu_seqlens, const float* h0, void* y, float* ht, void* workspace,
                            size_t workspace_bytes, void* stream) {
  ckda::ScanArgs a;
  ckda_status_t st = validate_scan(d, cu_seqlens, kScanFwd, &a);
  if (st != CKDA_OK) return st;
  const ScanSizes s = scan_sizes(d);
  const bool some = s.tokens > 0;
  const uint32_t el = static_cast<uint32_t>(s.es);
  const Tensor ts[] = {{rows_range("x", x, s.tokens, a.sx, d->D, s.es), false, some, el},
                       {rows_range("dt", dt, s.tokens, a.sdt, d->D, s.es), false, some, el},
                       {range("A", A, A ? s.A : 0), false, true},
                       {rows_range("B", B, s.tokens, a.sb, s.bc, s.es), false, some, el},
                       {rows_range("C", C, s.tokens, a.sc, s.bc, s.es), false, some, el},
                       {range("D", D, D ? s.vec : 0), false, false},
                       {rows_range("z", z, s.tokens, a.sz, d->D, s.es), false, false, el},
                       {range("dt_bias", dt_bias, dt_bias ? s.vec : 0), false, false},
                       {range("h0", h0, h0 ? s.state : 0), false, false},
                       {rows_range("y", y, s.tokens, d->D, d->D, s.es), true, some},
                       {range("ht", ht, ht ? s.state : 0), true, false}};
  if ((st = check_tensors(ts, 11, 8, 10)) != CKDA_OK) return st;
  if ((st = no_output_on(ts, 11, cu_seqlens, d->num_seqs)) != CKDA_OK) return st;
  const size_t need = d->num_seqs == 0 ? 0 : ckda::scan_fwd_workspace(a);
  if ((st = check_workspace(ts, 11, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  if (d->num_seqs == 0) return ok();
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.Bm = B;
  a.Cm = C;
  a.Dv = D;
  a.z = z;
  a.bias = dt_bias;
  a.h0 = h0;
  a.y = y;
  a.ht = ht;
  a.vec = scan_vec(a, s.es);
  return from_hip(ckda::launch_scan_fwd(a, d->io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_scan_bwd(const ckda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                            const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                            const int32_t* cu_seqlens, const float* h0, const void* dy, const float* dht, void* dx,
                            void* ddt, float* dA, void* dB, void* dC, float* dD, void* dz, float* ddt_bias,
                            float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  ckda::ScanArgs a;
  ckda_status_t st = validate_scan(d, cu_seqlens, kScanBwd, &a);
  if (st != CKDA_OK) return st;
  const ScanSizes s = scan_sizes(d);
  const bool some = s.tokens > 0;
  if (some && (z == nullptr) != (dz == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "dz is given exactly with z");
  if ((D == nullptr) != (dD == nullptr)) return fail(CKDA_ERR_INVALID_ARGUMENT, "dD is given exactly with D");
  if ((dt_bias == nullptr) != (ddt_bias == nullptr))
    return fail(CKDA_ERR_INVALID_ARGUMENT, "ddt_bias is given exactly with dt_bias");
  const uint32_t el = static_cast<uint32_t>(s.es);
  const Tensor ts[] = {{rows_range("x", x, s.tokens, a.sx, d->D, s.es), false, some, el},
                       {rows_range("dt", dt, s.tokens, a.sdt, d->D, s.es), false, some, el},
                       {range("A", A, A ? s.A : 0), false, true},
                       {rows_range("B", B, s.tokens, a.sb, s.bc, s.es), false, some, el},
                       {rows_range("C", C, s.tokens, a.sc, s.bc, s.es), false, some, el},
                       {range("D", D, D ? s.vec : 0), false, false},
                       {rows_range("z", z, s.tokens, a.sz, d->D, s.es), false, false, el},
                       {range("dt_bias", dt_bias, dt_bias ? s.vec : 0), false, false},
                       {range("h0", h0, h0 ? s.state : 0), false, false},
                       {rows_range("dy", dy, s.tokens, d->D, d->D, s.es), false, some},
                       {range("dht", dht, dht ? s.state : 0), false, false},
                       {rows_range("dx", dx, s.tokens, d->D, d->D, s.es), true, some},
                       {rows_range("ddt", ddt, s.tokens, d->D, d->D, s.es), true, some},
                       {range("dA", dA, dA ? s.A : 0), true, true},
                       {rows_range("dB", dB, s.tokens, s.bc, s.bc, s.es), true, some},
                       {rows_range("dC", dC, s.tokens, s.bc, s.bc, s.es), true, some},
                       {range("dD", dD, dD ? s.vec : 0), true, false},
                       {rows_range("dz", dz, s.tokens, d->D, d->D, s.es), true, false},
                       {range("ddt_bias", ddt_bias, ddt_bias ? s.vec : 0), true, false},
                       {range("dh0", dh0, dh0 ? s.state : 0), true, false}};
  if ((st = check_tensors(ts, 20)) != CKDA_OK) return st;
  if ((st = no_output_on(ts, 20, cu_seqlens, d->num_seqs)) != CKDA_OK) return st;
  const size_t need = ckda::scan_bwd_workspace(a);
  if ((st = check_workspace(ts, 20, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.Bm = B;
  a.Cm = C;
  a.Dv = D;
  a.z = z;
  a.bias = dt_bias;
  a.h0 = h0;
  a.dy = dy;
  a.dht = dht;
  a.dx = dx;
  a.ddt = ddt;
  a.dA = dA;
  a.dB = dB;
  a.dC = dC;
  a.dD = dD;
  a.dz = dz;
  a.dbias = ddt_bias;
  a.dh0 = dh0;
  a.vec = scan_vec(a, s.es);
  return from_hip(ckda::launch_scan_bwd(a, d->io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_scan_step(const ckda_scan_desc_t* d, const void* x, const void* dt, const float* A,
                             const void* B, const void* C, const float* D, const void* z, const float* dt_bias,
                             const float* h0, float* ht, void* y, void* stream) {
  if (d && d->B == 0 && d->num_seqs == 0) return ok();
  ckda::ScanArgs a;
  ckda_status_t st = validate_scan(d, nullptr, kScanStep, &a);
  if (st != CKDA_OK) return st;
  if (d->T != 1) return fail(CKDA_ERR_INVALID_ARGUMENT, "T=%d must be 1", d->T);
  const ScanSizes s = scan_sizes(d);
  if (s.state > (int64_t(1) << 33))
    return fail(CKDA_ERR_UNSUPPORTED, "N * D * S exceeds 2^31 for one decode launch");
  const uint32_t el = static_cast<uint32_t>(s.es);
  const Tensor ts[] = {{rows_range("x", x, s.tokens, a.sx, d->D, s.es), false, true, el},
                       {rows_range("dt", dt, s.tokens, a.sdt, d->D, s.es), false, true, el},
                       {range("A", A, s.A), false, true},
                       {rows_range("B", B, s.tokens, a.sb, s.bc, s.es), false, true, el},
                       {rows_range("C", C, s.tokens, a.sc, s.bc, s.es), false, true, el},
                       {range("D", D, D ? s.vec : 0), false, false},
                       {rows_range("z", z, s.tokens, a.sz, d->D, s.es), false, false, el},
                       {range("dt_bias", dt_bias, dt_bias ? s.vec : 0), false, false},
                       {range("h0", h0, s.state), false, true},
                       {range("ht", ht, s.state), true, true},
                       {rows_range("y", y, s.tokens, d->D, d->D, s.es), true, true}};
  if ((st = check_tensors(ts, 11, 8, 9)) != CKDA_OK) return st;
  a.x = x;
  a.dt = dt;
  a.A = A;
  a.Bm = B;
  a.Cm = C;
  a.Dv = D;
  a.z = z;
  a.bias = dt_bias;
  a.h0 = h0;
  a.ht = ht;
  a.y = y;
  return from_hip(ckda::launch_scan_step(a, d->io_dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// ---- layer norm ---------------------------------------------------------------------
extern "C" {

size_t ckda_layer_norm_bwd_workspace_size(int64_t rows, int32_t d, int32_t io_dtype) {
  if (rows <= 0 || d <= 0 || d > 16384) return 0;
  if (io_dtype != CKDA_DTYPE_BF16 && io_dtype != CKDA_DTYPE_F32) return 0;
  return ckda::layer_norm_bwd_workspace(rows, d);
}

ckda_status_t ckda_layer_norm(int64_t rows, int32_t d, int32_t io_dtype, float eps, const void* x, const void* r,
                              const float* w, const float* b, void* n, void* h, void* stream) {
  ckda_status_t st = validate_norm(rows, d, io_dtype, CKDA_NORM_GATE_NONE, eps, nullptr);
  if (st != CKDA_OK) return st;
  if ((r == nullptr) != (h == nullptr) && rows > 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "h is given exactly with r");
  const int64_t by = rows * d * elem_bytes(io_dtype), v = 4 * static_cast<int64_t>(d);
  const bool some = rows > 0;
  // h may be the very buffer of r or of x: a row is read before it is written
  const bool same = h != nullptr && (h == r || h == x);
  const Tensor ts[] = {{range("x", x, x ? by : 0), false, some}, {range("r", r, r ? by : 0), false, false},
                       {range("w", w, w ? v : 0), false, false}, {range("b", b, b ? v : 0), false, false},
                       {range("n", n, n ? by : 0), true, some},  {range("h", h, h ? by : 0), true, false}};
  if ((st = check_tensors(ts, 6, same && h == x ? 0 : 1, 5)) != CKDA_OK) return st;
  if (rows == 0) return ok();
  const ckda::LayerNormArgs a{rows, d, eps, x, r, w, b, n, h};
  return from_hip(ckda::launch_layer_norm(a, io_dtype, static_cast<hipStream_t>(stream)));
}

ckda_status_t ckda_layer_norm_bwd(int64_t rows, int32_t d, int32_t io_dtype, float eps, const void* x,
                                  const float* w, const void* dn, const void* dh, void* dx, float* dw, float* db,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  ckda_status_t st = validate_norm(rows, d, io_dtype, CKDA_NORM_GATE_NONE, eps, nullptr);
  if (st != CKDA_OK) return st;
  if (rows == 0)
    return fail(CKDA_ERR_INVALID_ARGUMENT, "no rows: the sums over rows would not be written");
  if ((w == nullptr) != (dw == nullptr)) return fail(CKDA_ERR_INVALID_ARGUMENT, "dw is given exactly with w");
  const int64_t by = rows * d * elem_bytes(io_dtype), v = 4 * static_cast<int64_t>(d);
  const Tensor ts[] = {{range("x", x, x ? by : 0), false, true},   {range("w", w, w ? v : 0), false, false},
                       {range("dn", dn, dn ? by : 0), false, true}, {range("dh", dh, dh ? by : 0), false, false},
                       {range("dx", dx, dx ? by : 0), true, true}, {range("dw", dw, dw ? v : 0), true, false},
                       {range("db", db, db ? v : 0), true, false}};
  if ((st = check_tensors(ts, 7)) != CKDA_OK) return st;
  const size_t need = ckda_layer_norm_bwd_workspace_size(rows, d, io_dtype);
  if ((st = check_workspace(ts, 7, workspace, workspace_bytes, need)) != CKDA_OK) return st;
  const ckda::LayerNormArgs a{rows, d, eps, x, nullptr, w, nullptr, nullptr, nullptr};
  const ckda::LayerNormGrads g{dn, dh, dx, dw, db, nullptr};
  return from_hip(ckda::launch_layer_norm_bwd(a, g, io_dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

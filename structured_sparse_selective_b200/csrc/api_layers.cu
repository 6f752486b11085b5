// C-ABI entry points of the layers beside the scan: the norm and rotation of queries and
// keys, and the gated delta rule. Validation, workspace layout and dispatch; the
// contract is in include/pdssm.h.
#include <math.h>

#include <algorithm>

#include "api_util.h"
#include "delta_chunk.cuh"
#include "launch.h"
#include "pdssm.h"

using namespace pdssm;

namespace {

// Makes the stream's device current for the call and puts the caller's back after it.
// A capturing stream may not be asked for its device (the question ends the capture):
// there the caller has that device current, as the capture needs it anyway.
class OnDevice {
 public:
  explicit OnDevice(cudaStream_t stream) {
    if (stream == nullptr) return;
    cudaStreamCaptureStatus capturing;
    if (cudaStreamIsCapturing(stream, &capturing) != cudaSuccess) {
      status_ = PDSSM_ERR_CUDA;
      return;
    }
    if (capturing != cudaStreamCaptureStatusNone) return;
    int dev = -1;
    if (cudaStreamGetDevice(stream, &dev) != cudaSuccess || cudaGetDevice(&before_) != cudaSuccess) {
      status_ = PDSSM_ERR_CUDA;
      return;
    }
    if (before_ == dev) return;
    if (cudaSetDevice(dev) == cudaSuccess) changed_ = true;
    else status_ = PDSSM_ERR_CUDA;
  }
  ~OnDevice() {
    if (changed_) cudaSetDevice(before_);
  }
  pdssm_status status() const { return status_; }

 private:
  int before_ = 0;
  bool changed_ = false;
  pdssm_status status_ = PDSSM_OK;
};

bool real_type(int t) { return t == PDSSM_F32 || t == PDSSM_BF16; }

pdssm_status check_norm(const pdssm_norm_problem *pb, int64_t *rows) {
  if (!pb) return PDSSM_ERR_INVALID_ARG;
  if (pb->batch < 0 || pb->seqlen < 0 || pb->q_heads < 0 || pb->k_heads < 0 || pb->N < 1 || pb->rot < 0 ||
      (pb->rot & 1) || pb->rot > pb->N || !(pb->eps >= 0.f) || !(pb->eps < INFINITY) || pb->flags != 0 ||
      (pb->interleaved != 0 && pb->interleaved != 1) || (pb->mode != PDSSM_NORM_RMS && pb->mode != PDSSM_NORM_L2))
    return PDSSM_ERR_INVALID_ARG;
  if (pb->N > PDSSM_MAX_N || !real_type(pb->io_t) || pb->q_heads > 65535 || pb->k_heads > 65535 ||
      pb->seqlen > INT32_MAX)
    return PDSSM_ERR_UNSUPPORTED;
  int64_t n;
  if (!mul_ok(pb->batch, pb->seqlen, rows) || !mul_ok(*rows, 65535 * PDSSM_MAX_N * 4, &n)) return PDSSM_ERR_UNSUPPORTED;
  return PDSSM_OK;
}

size_t norm_bwd_bytes(const pdssm_norm_problem *pb, int64_t rows) {
  return rows ? align256((size_t)2 * qk_norm_bwd_blocks(rows) * pb->N * 4) : 0;
}

pdssm_status run_norm(const pdssm_norm_problem *pb, QkNormArgs &a, int64_t rows, bool bwd, cudaStream_t cs) {
  a.rows = rows; a.seqlen = pb->seqlen; a.heads[0] = pb->q_heads; a.heads[1] = pb->k_heads; a.N = pb->N;
  a.io_t = pb->io_t; a.rot = pb->rot; a.interleaved = pb->interleaved;
  a.l2 = pb->mode == PDSSM_NORM_L2;
  a.eps = pb->eps;
  return cuda_status(launch_qk_norm(a, bwd, cs));
}

struct DeltaPlan {
  int64_t rows, slices, Pp, C, nC;
  bool chunked, by_rows;  // by chunks on the tensor cores, or in fp32
  size_t o_carry, o_xcarry, o_e, o_du, o_dyy, o_rec, o_heads, bytes;
};

constexpr size_t kErrBytes = 256;

// Whether a problem goes by chunks of 64 steps on the tensor cores, or step by step: bf16
// inputs, and as measured (us; steps, chunks; N = P = 64 with 256 sequences, 128 x 64 with 2,048):
//   forward   256: 32 steps 25, 29; 48 steps 35, 29; 64 steps 45, 27
//             2,048: 8 steps 167, 187; 16 steps 235, 189; 32 steps 353, 191
//   backward  256: 8 steps 56, 56; 16 steps 64, 57; 64 steps 140, 53
//             2,048: 8 steps 829, 431
// A chunk costs the same however few of its steps there are; steps cost their number, more
// where four sequences or more share an SM. The rule does not look at P, nor at N below 64; there it is
// not always the faster one:
//   forward   N = P = 32: 256: 64 steps 16, 31; 2,048: 16 steps 35, 151; 64 steps 86, 154
//             64 x 8: 2,048: 16 steps 35, 151; 64 steps 95, 152.  128 x 128: 256: 16 steps 62, 43; 64 steps 189, 43
//   backward  N = P = 32: 2,048: 16 steps 198, 321; 32 steps 265, 330.  64 x 8: 2,048: 32 steps 263, 327
//             128 x 128: 256: 4 steps 174, 108; 32 steps 267, 114
bool chunks_apply(const pdssm_delta_problem *pb, bool bwd) {
  if (pb->in_t != PDSSM_BF16 || (pb->flags & PDSSM_FLAG_REFERENCE_PATH)) return false;
  if (bwd) return pb->seqlen > 8;
  return pb->seqlen > (pb->batch * pb->heads >= 4 * 148 ? 12 : 40);
}

// The same for fp32 inputs and chunks of 32 steps in fp32 (us; steps, chunks; S sequences x heads, N = P):
//   forward   N = 64:  S = 8: 128 steps 30, 29; 512 steps 93, 46.  S = 64: 128 steps 31, 40; 512 steps 103, 90.
//                      S = 128: 512 steps 126, 156.  S = 1024: 512 steps 902, 969.
//             N = 128: S = 64: 64 steps 46, 50; 128 steps 85, 82.  S = 256: 128 steps 308, 240; 512 steps 1205, 864.
//   backward  N = 64:  S = 64: 64 steps 46, 37; 128 steps 80, 53; 512 steps 268, 151.  S = 256: 512 steps 474, 491.
//             N = 128: S = 64: 64 steps 92, 80; 512 steps 638, 450.  S = 256: 512 steps 2033, 1433.
//   forward   N = 32:  S = 8: 128 steps 19, 17; 512 steps 60, 25.  S = 64: 128 steps 19, 21; 512 steps 62, 39.
//                      S = 256: 512 steps 80, 115.  S = 1024: 512 steps 303, 384.
//   backward  N = 32:  S = 64: 64 steps 35, 35; 512 steps 179, 129.  S = 256: 512 steps 495, 466.
// A step's chain of shuffles is what few sequences wait for; many fill the SMs either way, and then
// steps do fewer FMAs, unless a head is so large that its columns do not fit in a few registers a lane.
// The rule does not look at P: with N = 128 and P = 8 (S = 256: 512 steps 176, 251; S = 1024: 680, 1084) steps would
// be the faster ones, with N = 32 and P = 128 (S = 64: 512 steps 80, 86) it is even.
bool rows_apply(const pdssm_delta_problem *pb, bool bwd) {
  if (pb->in_t != PDSSM_F32 || (pb->flags & PDSSM_FLAG_REFERENCE_PATH)) return false;
  if (pb->N > 64) return pb->seqlen > (bwd ? 64 : 96);
  const int64_t slices = pb->batch * pb->heads;
  return bwd ? slices <= 148 && pb->seqlen > 96 : slices <= 64 && pb->seqlen > 256;
}

pdssm_status plan_delta(const pdssm_delta_problem *pb, bool bwd, DeltaPlan *pl) {
  if (!pb) return PDSSM_ERR_INVALID_ARG;
  if (pb->batch < 0 || pb->seqlen < 0 || pb->heads < 1 || pb->qk_heads < 1 || pb->heads % pb->qk_heads ||
      pb->N < 1 || pb->P < 1 || !isfinite(pb->scale) ||
      (pb->flags & ~(PDSSM_FLAG_REFERENCE_PATH | PDSSM_FLAG_SHORT_WAITS)))
    return PDSSM_ERR_INVALID_ARG;
  if (pb->N > PDSSM_MAX_N || pb->P > PDSSM_MAX_P || pb->batch > 65535 || pb->heads > 65535 ||
      !real_type(pb->in_t) || !real_type(pb->gate_t) || pb->seqlen > (int64_t)1 << 35)
    return PDSSM_ERR_UNSUPPORTED;
  DeltaPlan p;
  p.Pp = (pb->P + 3) / 4 * 4;
  int64_t bytes;
  p.slices = pb->batch * pb->heads;
  // the largest arrays: states of up to 64 KiB a chunk of 32 steps (with the record of 64 steps no
  // more than 8 KiB a step), rows of Pp floats a step
  if (!mul_ok(pb->batch, pb->seqlen, &p.rows) || !mul_ok(p.slices, (pb->seqlen + kChunk) * 8192, &bytes))
    return PDSSM_ERR_UNSUPPORTED;
  p.chunked = chunks_apply(pb, bwd);
  p.by_rows = rows_apply(pb, bwd);
  p.C = p.chunked ? kChunk : delta_grad_chunk();
  p.nC = (pb->seqlen + p.C - 1) / p.C;
  const size_t records = p.chunked ? (size_t)(p.slices * p.nC * delta_record_bytes(bwd)) : 0;
  size_t o = p.chunked || p.by_rows || bwd ? kErrBytes : 0;
  if (bwd) {
    // error word, states (chunked: one more a sequence), adjoints, e, du; chunked: <dy, y> and the records
    const size_t state = (size_t)(pb->N * p.Pp) * 4, steps = (size_t)(p.rows * pb->heads * p.Pp) * 4;
    p.o_carry = o; o = align256(o + (size_t)(p.slices * (p.nC + (p.chunked ? 1 : 0))) * state);
    p.o_xcarry = o; o = align256(o + (size_t)(p.slices * p.nC) * state);
    p.o_e = o; o = align256(o + steps);
    p.o_du = o; o = align256(o + steps);
    p.o_dyy = o; o = align256(o + (p.chunked ? (size_t)(p.rows * pb->heads) * 16 : 0));
  }
  p.o_rec = o; o = align256(o + (p.by_rows ? (size_t)(pb->batch * pb->qk_heads * p.nC * delta_rows_key_bytes(pb->N)) : records));
  p.o_heads = o; o = align256(o + (p.by_rows ? (size_t)(p.slices * p.nC * delta_rows_head_bytes(bwd)) : 0));
  p.bytes = o;
  *pl = p;
  return PDSSM_OK;
}

uint64_t wait_limit(const pdssm_delta_problem *pb) {
  return (pb->flags & PDSSM_FLAG_SHORT_WAITS) ? 1000ull : 2000000000ull;
}

DeltaArgs delta_args(const pdssm_delta_problem *pb, const DeltaPlan &p) {
  DeltaArgs a{};
  a.Bt = pb->batch; a.L = pb->seqlen; a.H = pb->heads; a.Hk = pb->qk_heads; a.N = pb->N; a.P = pb->P;
  a.Pp = p.Pp; a.C = p.C; a.nC = p.nC;
  a.in_t = pb->in_t; a.gate_t = pb->gate_t;
  a.scale = pb->scale;
  return a;
}

// The error word, cleared, of a call that launches nothing.
pdssm_status clear_error(uint32_t *err, cudaStream_t cs) {
  return !err || cudaMemsetAsync(err, 0, 4, cs) == cudaSuccess ? PDSSM_OK : PDSSM_ERR_CUDA;
}

// Records and wait limit of the kernels with roles, and their error word cleared.
pdssm_status use_records(const pdssm_delta_problem *pb, const DeltaPlan &p, bool bwd, void *workspace, DeltaArgs &a, cudaStream_t cs) {
  char *base = static_cast<char *>(workspace);
  a.records = reinterpret_cast<uint8_t *>(base + p.o_rec);
  a.rec_bytes = delta_record_bytes(bwd);
  a.keys = reinterpret_cast<float *>(base + p.o_rec);
  a.heads = reinterpret_cast<float *>(base + p.o_heads);
  a.wait_ns = wait_limit(pb);
  return clear_error(a.err, cs);
}

}  // namespace

extern "C" {

pdssm_status pdssm_qk_norm(const pdssm_norm_problem *pb, const void *q, const void *k, const float *wq,
                           const float *wk, const float *inv_freq, const int32_t *positions, void *q_out,
                           void *k_out, pdssm_stream_t stream) {
  int64_t rows;
  pdssm_status st = check_norm(pb, &rows);
  if (st != PDSSM_OK) return st;
  if (rows == 0 || pb->q_heads + pb->k_heads == 0) return PDSSM_OK;
  const size_t es = dtype_size(pb->io_t);
  if ((pb->q_heads && (!q || !q_out)) || (pb->k_heads && (!k || !k_out)) || (pb->rot && !inv_freq))
    return PDSSM_ERR_INVALID_ARG;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(q_out, es) || !aligned(k_out, es) || !aligned(wq, 4) ||
      !aligned(wk, 4) || !aligned(inv_freq, 4) || !aligned(positions, 4))
    return PDSSM_ERR_INVALID_ARG;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  OnDevice on(cs);
  if (on.status() != PDSSM_OK) return on.status();
  QkNormArgs a{};
  a.x[0] = q; a.x[1] = k; a.out[0] = q_out; a.out[1] = k_out; a.w[0] = wq; a.w[1] = wk;
  a.inv_freq = inv_freq; a.positions = positions;
  return run_norm(pb, a, rows, false, cs);
}

pdssm_status pdssm_qk_norm_bwd_workspace_size(const pdssm_norm_problem *pb, size_t *bytes) {
  if (!bytes) return PDSSM_ERR_INVALID_ARG;
  int64_t rows;
  pdssm_status st = check_norm(pb, &rows);
  if (st != PDSSM_OK) return st;
  *bytes = norm_bwd_bytes(pb, rows);
  return PDSSM_OK;
}

pdssm_status pdssm_qk_norm_bwd(const pdssm_norm_problem *pb, const void *q, const void *k, const float *wq,
                               const float *wk, const float *inv_freq, const int32_t *positions,
                               const void *dq_out, const void *dk_out, void *dq, void *dk, float *dwq, float *dwk,
                               void *workspace, size_t workspace_bytes, pdssm_stream_t stream) {
  int64_t rows;
  pdssm_status st = check_norm(pb, &rows);
  if (st != PDSSM_OK) return st;
  const size_t es = dtype_size(pb->io_t);
  if ((dwq && !wq) || (dwk && !wk)) return PDSSM_ERR_INVALID_ARG;
  if (rows && ((pb->q_heads && (!q || !dq_out || !dq)) || (pb->k_heads && (!k || !dk_out || !dk)) || (pb->rot && !inv_freq)))
    return PDSSM_ERR_INVALID_ARG;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(dq_out, es) || !aligned(dk_out, es) || !aligned(dq, es) ||
      !aligned(dk, es) || !aligned(wq, 4) || !aligned(wk, 4) || !aligned(inv_freq, 4) || !aligned(positions, 4) ||
      !aligned(dwq, 4) || !aligned(dwk, 4) || !aligned(workspace, 16))
    return PDSSM_ERR_INVALID_ARG;
  if ((dwq || dwk) && rows && (!workspace || workspace_bytes < norm_bwd_bytes(pb, rows))) return PDSSM_ERR_WORKSPACE;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  OnDevice on(cs);
  if (on.status() != PDSSM_OK) return on.status();
  if (rows == 0 || pb->q_heads + pb->k_heads == 0) {  // no tokens: nothing reaches the weights
    if (dwq && cudaMemsetAsync(dwq, 0, pb->N * 4, cs) != cudaSuccess) return PDSSM_ERR_CUDA;
    if (dwk && cudaMemsetAsync(dwk, 0, pb->N * 4, cs) != cudaSuccess) return PDSSM_ERR_CUDA;
    return PDSSM_OK;
  }
  QkNormArgs a{};
  a.x[0] = q; a.x[1] = k; a.dy[0] = dq_out; a.dy[1] = dk_out; a.out[0] = dq; a.out[1] = dk;
  a.w[0] = wq; a.w[1] = wk; a.dw[0] = dwq; a.dw[1] = dwk;
  a.inv_freq = inv_freq; a.positions = positions;
  a.part = static_cast<float *>(workspace);
  return run_norm(pb, a, rows, true, cs);
}

pdssm_status pdssm_delta_workspace_size(const pdssm_delta_problem *pb, size_t *bytes) {
  if (!bytes) return PDSSM_ERR_INVALID_ARG;
  DeltaPlan p;
  pdssm_status st = plan_delta(pb, false, &p);
  if (st != PDSSM_OK) return st;
  *bytes = p.bytes;
  return PDSSM_OK;
}

pdssm_status pdssm_delta_fwd(const pdssm_delta_problem *pb, const void *q, const void *k, const void *v,
                             const void *g, const void *beta, const int32_t *lengths, const float *h0, void *y,
                             float *h_final, void *workspace, size_t workspace_bytes, pdssm_stream_t stream) {
  DeltaPlan p;
  pdssm_status st = plan_delta(pb, false, &p);
  if (st != PDSSM_OK) return st;
  const size_t es = dtype_size(pb->in_t), gs = dtype_size(pb->gate_t);
  if (p.rows * pb->heads > 0 && (!q || !k || !v || !g || !beta || !y)) return PDSSM_ERR_INVALID_ARG;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(y, es) || !aligned(g, gs) ||
      !aligned(beta, gs) || !aligned(lengths, 4) || !aligned(h0, 4) || !aligned(h_final, 4) || !aligned(workspace, 16))
    return PDSSM_ERR_INVALID_ARG;
  if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return PDSSM_ERR_WORKSPACE;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  OnDevice on(cs);
  if (on.status() != PDSSM_OK) return on.status();
  // a workspace larger than needed has the word too
  uint32_t *err = workspace_bytes >= 4 ? static_cast<uint32_t *>(workspace) : nullptr;
  if (p.slices == 0) return clear_error(err, cs);
  DeltaArgs a = delta_args(pb, p);
  a.err = err;
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.lengths = lengths; a.h0 = h0; a.y = y; a.h_final = h_final;
  if (!p.chunked && !p.by_rows) return cuda_status(launch_delta_steps(a, cs));
  if ((st = use_records(pb, p, false, workspace, a, cs)) != PDSSM_OK) return st;
  if (p.by_rows) return cuda_status(launch_delta_rows(a, false, cs));
  if ((st = cuda_status(launch_delta_prep(a, false, cs))) != PDSSM_OK) return st;
  return cuda_status(launch_delta_chunk(a, cs));
}

pdssm_status pdssm_delta_bwd_workspace_size(const pdssm_delta_problem *pb, size_t *bytes) {
  if (!bytes) return PDSSM_ERR_INVALID_ARG;
  DeltaPlan p;
  pdssm_status st = plan_delta(pb, true, &p);
  if (st != PDSSM_OK) return st;
  *bytes = p.bytes;
  return PDSSM_OK;
}

pdssm_status pdssm_delta_bwd(const pdssm_delta_problem *pb, const void *q, const void *k, const void *v,
                             const void *g, const void *beta, const int32_t *lengths, const float *h0, const void *dy,
                             const float *dh_final, void *dq, void *dk, void *dv, void *dg, void *dbeta, float *dh0,
                             void *workspace, size_t workspace_bytes, pdssm_stream_t stream) {
  DeltaPlan p;
  pdssm_status st = plan_delta(pb, true, &p);
  if (st != PDSSM_OK) return st;
  const size_t es = dtype_size(pb->in_t), gs = dtype_size(pb->gate_t);
  if (p.rows * pb->heads > 0 &&
      (!q || !k || !v || !g || !beta || !dy || !dq || !dk || !dv || !dg || !dbeta))
    return PDSSM_ERR_INVALID_ARG;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(dy, es) || !aligned(dq, es) ||
      !aligned(dk, es) || !aligned(dv, es) || !aligned(g, gs) || !aligned(beta, gs) || !aligned(dg, gs) ||
      !aligned(dbeta, gs) || !aligned(lengths, 4) || !aligned(h0, 4) || !aligned(dh_final, 4) || !aligned(dh0, 4) ||
      !aligned(workspace, 16))
    return PDSSM_ERR_INVALID_ARG;
  if (p.bytes && (!workspace || workspace_bytes < p.bytes)) return PDSSM_ERR_WORKSPACE;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  OnDevice on(cs);
  if (on.status() != PDSSM_OK) return on.status();
  if (p.slices == 0) return clear_error(static_cast<uint32_t *>(workspace), cs);
  DeltaArgs a = delta_args(pb, p);
  a.err = static_cast<uint32_t *>(workspace);
  char *base = static_cast<char *>(workspace);
  a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.lengths = lengths; a.h0 = h0; a.dy = dy; a.dh_final = dh_final;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
  a.carry = reinterpret_cast<float *>(base + p.o_carry);
  a.xcarry = reinterpret_cast<float *>(base + p.o_xcarry);
  a.e = reinterpret_cast<float *>(base + p.o_e);
  a.du = reinterpret_cast<float *>(base + p.o_du);
  if ((p.chunked || p.by_rows) && (st = use_records(pb, p, true, workspace, a, cs)) != PDSSM_OK) return st;
  if (p.chunked) {
    a.dyy = reinterpret_cast<float *>(base + p.o_dyy);
    if ((st = cuda_status(launch_delta_prep(a, true, cs))) != PDSSM_OK) return st;
    if ((st = cuda_status(launch_delta_chunk_both(a, cs))) != PDSSM_OK) return st;
    return cuda_status(launch_delta_chunk_grad(a, cs));
  }
  st = cuda_status(p.by_rows ? launch_delta_rows(a, true, cs) : launch_delta_steps_both(a, cs));
  if (st != PDSSM_OK) return st;
  if (p.rows > 0) st = cuda_status(launch_delta_grad(a, cs));
  return st;
}

}  // extern "C"

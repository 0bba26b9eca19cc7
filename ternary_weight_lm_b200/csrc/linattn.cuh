// Linear attention with a decay for each head: the sweeps that its forward and backward are made
// of, and their launchers.  Internal to libmmf.so.
#pragma once

#include "kernels.cuh"

namespace mmf {

// One sweep over the tokens of every sequence and head.  With S the state [dk x dv]:
//   forwards    S = gamma S + a k_t v_t^T,  o_t = b S^T q_t
//   backwards   (last token first)  R = U + a k_t v_t^T,  o_t = b R^T q_t,  U = gamma R
// k_t and q_t have dk values, v_t and o_t dv.  s0 (or nullptr: zero) is S or U before the first
// token taken, sT (or nullptr) receives it after the last.  Element (i, j) of sequence b, head h
// of s0 and sT is at ((b H + h) dk dv) + i s_key + j s_val.
struct LinSweep {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h, o_t, o_h;   // element strides of a token and of a head
  int dk, dv;
  float a, b;
  int backwards;
  const float* s0;
  float* sT;
  int s_key, s_val;
  float* seg;      // workspace: one state [dk x dv] for each (item, head), or nullptr (unsplit)
};

constexpr int kMaxSweeps = 3;

// The kernels of a sweep: token by token (every type and size), chunks of 64 tokens on mma.sync, chunks
// of 128 on tcgen05.
enum LinForm { kLinTokens, kLinMma, kLinTc };

// A call.  Sequence b has the tokens [cu[b], cu[b + 1]) or, without cu, [b T / B, (b + 1) T / B).
// Work items: every sequence is cut into segments of `seg_len` tokens in the sweep's order (the
// last one is shorter); item x of n_items names a sequence and a segment, items past the last are
// empty.
struct LinCall {
  LinSweep sw[kMaxSweeps];
  int n_sweeps;
  LinForm form;            // of every sweep
  int dt;                  // InDType of q, k, v, o
  int64_t T;
  int B;
  int H;
  const int32_t* cu;
  const float* log_decay;  // [H]
  int64_t seg_len;
  int64_t n_items;
  int clear;               // zeros for the rows of tokens outside the sequences
  int split;               // segments start from states found by a pass over k and v first
  unsigned* status;
};

// Which form a call of these sizes, type and strides takes (token and head of q, k, v and, backwards,
// of the outputs' gradient).
LinForm lin_form(int H, int dk, int dv, int dt, int n_sweeps, const int64_t (*strides)[2]);
// Segment length for a call of these sizes and form (a function of them alone), the number of items
// and whether the sequences are split.
void lin_plan(int64_t T, int64_t B, bool ragged, int H, int dk, int dv, LinForm form, int n_sweeps,
              int64_t* seg_len, int64_t* n_items, int* split);
size_t lin_seg_bytes(int64_t n_items, int H, int dk, int dv);

cudaError_t launch_linattn(const LinCall& c, cudaStream_t s);

cudaError_t launch_lin_mma(const LinCall& c, cudaStream_t s);
// The second pass of a split: every segment's start state from the segments' own contributions.
cudaError_t launch_lin_join(const LinCall& c, cudaStream_t s);

cudaError_t launch_lin_tc(const LinCall& c, cudaStream_t s);

// One token of each sequence: state [rows x H x dk x dv] updated in place, o = scale S^T q.
// q, k, v, o: [B x H x d] with strides of a sequence and of a head.  slots (or nullptr: row b is
// state b): the state of each sequence; a slot outside [0, n_slots) or named before is skipped.
struct LinStep {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  int64_t q_b, q_h, k_b, k_h, v_b, v_h, o_b, o_h;
  int dt;
  int64_t B;
  int H, dk, dv;
  const float* log_decay;
  float scale;
  float* state;
  const int32_t* slots;
  int64_t n_slots;
  unsigned* status;
};
cudaError_t launch_linattn_step(const LinStep& c, cudaStream_t s);

}  // namespace mmf

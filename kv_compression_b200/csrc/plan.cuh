// plan.cuh -- the plan behind the opaque lca_plan of include/lca.h, shared by
// the library's translation units.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "lca.h"

struct lca_plan {
  int B, H, d_c, d_r;
  lca_dtype dt;
  int64_t max_L;
  int device;
  int num_sms;
  bool tc_shape;           // the tcgen05 kernel can take this shape
  bool pair_shape;         // the two-CTA tcgen05 kernel can take this shape (H % 128 == 0)
  int pair_clusters;       // two-CTA clusters resident at once on this device
  int64_t ws_slots;
  float* part_o;           // [ws_slots][H][d_c]
  float* part_mz;          // [ws_slots][H][2]
  int* meta;               // paged-decode metadata, lca::meta_ints(B, ws_slots) ints
  int* err;                // [2]: flags, where
  int last_site;           // where of the last error lca_get_device_error reported
  // options
  bool force_simt;
  int kernel_pref;         // 0: automatic, else the lca_plan_kernel code to use
  int num_ctas;
  uint64_t timeout_ns;
  int debug_skip_load;
  cudaEvent_t timing_event;  // recorded between the main and the combine kernel when set
  int64_t bias_rows;         // set only for the duration of an lca_decode_stored call
  float bias;
  // lca_decode_host staging (allocated on first use)
  void* st_qc;
  void* st_qr;
  void* st_c;
  void* st_k;
  float* st_out;
  int32_t* st_anc;
};

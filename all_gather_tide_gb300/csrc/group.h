// The group object behind tide_group_t.
#pragma once

#include <cstdint>
#include <mutex>

#include "../../include/tide.h"
#include "table_ring.h"
#include "tide_internal.h"

namespace tide {
constexpr int kMaxCeLanes = 8;  // helper streams for copy-engine work
}

struct tide_group {
    tide::Plan plan;
    uint32_t flags = 0;
    int device = 0;
    int sm_count = 0;
    int rs_ctas = 0, ag_ctas = 0;  // 0 = default
    int rs_variant = TIDE_RS_AUTO;
    int ag_variant = TIDE_AG_AUTO;
    uint64_t timeout_ns = tide::kDefaultTimeoutNs;
    uint32_t debug = 0;
    int* d_status = nullptr;  // device status word written by bounded waits that expire
    tide::RsSeg* d_rs = nullptr;
    int32_t* d_rs_piece = nullptr;  // piece index of every register-path chunk
    tide::RsSeg* d_rs_bulk = nullptr;
    int32_t* d_rs_bulk_piece = nullptr;  // piece index of every bulk chunk
    tide::RsSeg* d_rs_slots = nullptr;      // pieces of the summing step over staging slots
    int32_t* d_rs_slot_piece = nullptr;     // piece (0..P-1) of every chunk of one destination
    tide::AgSeg* d_ag_bulk = nullptr;
    tide::AgSeg* d_ag = nullptr;
    int32_t* d_ag_run = nullptr;  // run index of every register-path placement chunk
    tide::TableRing ring;
    int64_t last_ce_copies = 0;
    int32_t last_ce_uniform = 0;
    // copy-engine work is spread over `ce_lanes` streams forked from and joined back to the
    // caller's stream, so several copy engines run at once
    int ce_lanes = tide::kMaxCeLanes;  // measured on GB300: 1-D copies over 8 streams reach ~0.94 x HBM peak
    int ce_bands = 1;  // 2-D copies per parameter (bands of ranks)
    cudaStream_t lane_stream[tide::kMaxCeLanes] = {};
    cudaEvent_t lane_done[tide::kMaxCeLanes] = {};
    cudaEvent_t fork = nullptr;
    std::mutex mu;
};
